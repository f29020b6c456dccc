"""What stands on the target's side of a speculative round -- attention of many
candidates over the prompt that they share, log probabilities of the tokens
that a round emitted with the target's entropy and top alternatives, and the
loss that trains a draft on those alternatives, with its gradient -- as
measured cases: their inputs, their plain form, the framework's calls and a
64-bit form.

With ``own`` false, ``run`` computes an operator from elementary torch
operations; with ``own`` true it makes the framework's call.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the tiny chain's emitted tokens for one user, latency counts
        dict(name="logprobs_tiny", op="logprobs", B=1, T=5, P=5, V=1000, dt="f32", K=5, pad=0,
             temperature=1.0, tokens="all"),
        # a round of the large-vocabulary chain: what each sequence emitted
        # (the accepted drafts and one more), -1 behind it
        dict(name="logprobs_round", op="logprobs", B=256, T=8, P=8, V=128256, dt="bf16", K=5,
             pad=0, temperature=1.0, tokens="round"),
        # a round of the static tree: the rows are those of the accepted path
        dict(name="logprobs_tree", op="logprobs", B=32, T=25, P=6, V=32000, dt="bf16", K=1, pad=0,
             temperature=1.0, tokens="tree"),
        # scoring the tokens of long prompts
        dict(name="logprobs_prompt", op="logprobs", B=4, T=1024, P=1024, V=128256, dt="bf16",
             K=20, pad=0, temperature=1.0, tokens="all"),
        # a teacher's pass over training text: no given tokens, many
        # alternatives, an odd vocabulary in padded rows, a temperature
        dict(name="logprobs_teacher", op="logprobs", B=1, T=1000, P=1000, V=50257, dt="f32", K=64,
             pad=47, temperature=0.7, tokens="none"),
        # one short chain's rows, small vocabulary, latency
        dict(name="distill_tiny", op="distill", R=5, V=1000, dt="f32", K=8, temperature=1.0,
             tail=True, mode="both", weight=False),
        # a training step of a draft: loss and gradient at once
        dict(name="distill_train", op="distill", R=2048, V=128256, dt="bf16", K=64,
             temperature=1.0, tail=True, mode="both", weight=True),
        # held-out text: the loss alone, the teacher's weights normalised over its list
        dict(name="distill_eval", op="distill", R=1500, V=32000, dt="bf16", K=20, temperature=2.0,
             tail=False, mode="loss", weight=False),
        # the backward pass alone, after a forward pass that saved its row
        # statistics; odd vocabulary in packed rows
        dict(name="distill_backward", op="distill", R=777, V=40001, dt="f32", K=32,
             temperature=1.0, tail=True, mode="grad", weight=True),
        # one user's prompt with four candidate continuations, latency
        dict(name="prefix_one", op="prefix", N=1, W=4, Hq=32, Hkv=8, D=128, lo=1000, hi=1013,
             own_lo=1, own_hi=20, page=16, dt="bf16"),
        # a batch of the dynamic-tree workload's size and heads, all of it
        # behind one long document
        dict(name="prefix_document", op="prefix", N=1, W=128, Hq=64, Hkv=8, D=128, lo=32500,
             hi=32768, own_lo=1, own_hi=600, page=64, dt="bf16"),
        # several prompts, eight samples of each; small heads, fp16, pages of
        # no round size, some samples that have no slots of their own yet
        dict(name="prefix_samples", op="prefix", N=16, W=8, Hq=32, Hkv=8, D=64, lo=1500, hi=9000,
             own_lo=0, own_hi=300, page=20, dt="f16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "distill", "distill", "prefix", "prefix"])
    if op == "logprobs":
        V = _log_int(rng, 17, 128256)
        tokens = rng.choice(["all", "all", "round", "tree", "none"])
        T = _log_int(rng, 1, 60)
        B = _log_int(rng, 1, max(2, min(256, 250000000 // (T * V))))
        return dict(op="logprobs", B=B, T=T, P=rng.randint(1, min(T, 8)) if tokens == "tree" else T,
                    V=V, dt=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    K=min(V, rng.choice([0, 1, 2, 5, 20, 50, 100, 128])),
                    pad=rng.choice([0, 0, 1, 8, 47]), temperature=rng.choice([1.0, 1.0, 0.7, 2.0]),
                    tokens=tokens)
    if op == "distill":
        V = _log_int(rng, 129, 128256)
        return dict(op="distill", R=_log_int(rng, 1, max(2, min(4096, 130000000 // V))), V=V,
                    dt=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    K=rng.choice([1, 2, 8, 20, 50, 100, 128]),
                    temperature=rng.choice([1.0, 1.0, 0.7, 2.0]), tail=rng.random() < 0.6,
                    mode=rng.choice(["both", "both", "loss", "grad"]), weight=rng.random() < 0.6)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    D = rng.choice([64, 128])
    W = _log_int(rng, 1, 128)
    N = _log_int(rng, 1, max(1, 128 // W))
    hi = _log_int(rng, 17, max(18, min(131072, (1 << 35) // (W * N * Hkv * G * D),
                                       (1 << 27) // (N * Hkv * D))))
    own_hi = _log_int(rng, 1, 600)
    return dict(op="prefix", N=N, W=W, Hq=Hkv * G, Hkv=Hkv, D=D, lo=max(1, hi // rng.choice([1, 2, 8])),
                hi=hi, own_lo=rng.choice([0, 1, own_hi]), own_hi=own_hi,
                page=rng.choice([1, 8, 16, 20, 32, 64, 128]), dt=rng.choice(["bf16", "f16"]))


# ----------------------------------------------------------------- the inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(g, lo, hi, *shape):
    """From lo to hi, both possible."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _prepare_logprobs(c, g):
    B, T, P, V, K = c["B"], c["T"], c["P"], c["V"], c["K"]
    buf = torch.zeros(B, T, V + c["pad"], dtype=_DT[c["dt"]], device="cuda")
    logits = buf[:, :, :V]
    logits.copy_(_randn(g, B, T, V).mul_(3))
    rows = tokens = None
    if c["tokens"] != "none":
        # tokens as the target would draw them: the largest of logit + Gumbel noise
        u = torch.rand(B, T, V, generator=g, device="cuda").clamp_(1e-20, 1 - 1e-7)
        drawn = u.log_().neg_().log_().neg_().add_(logits).argmax(-1).to(torch.int32)
        p = torch.arange(P, device="cuda")
        if c["tokens"] == "tree":  # an increasing path of nodes from the root
            order = torch.rand(B, T, generator=g, device="cuda")
            order[:, 0] = -1
            path = order.argsort(1)[:, :P].sort(1).values
            some = p < _ints(g, 1, P, B)[:, None]
            rows = torch.where(some, path, -1).to(torch.int32)
            tokens = torch.where(some, drawn.gather(1, path), -1)
        else:
            tokens = drawn
            if c["tokens"] == "round":
                tokens = torch.where(p < _ints(g, 1, P, B)[:, None], drawn, -1)
    return dict(c=c, logits=logits, rows=rows, tokens=tokens)


def _prepare_distill(c, g):
    R, V, K = c["R"], c["V"], c["K"]
    x = _randn(g, R, V).mul_(3)
    logits = x.to(_DT[c["dt"]], copy=True)
    # a teacher near its student, at the same temperature
    x += _randn(g, R, V)
    top = torch.log_softmax(x.div_(c["temperature"]), -1).topk(K, -1)
    weight = None
    if c["weight"]:  # a mean over the rows, scaled up where the gradient's type ends early
        scale = (1 << 14 if c["dt"] == "f16" else 1) / R
        weight = torch.rand(R, generator=g, device="cuda").add_(0.5).mul_(scale)
    s = dict(c=c, logits=logits, token=top.indices.to(torch.int32), logprob=top.values.contiguous(),
             weight=weight, stat=None)
    if c["mode"] != "loss":
        s["grad"] = torch.empty_like(logits)
    if own and c["mode"] == "grad":  # saved by the forward pass
        import speculative_decoding_verification_vocab_gb300 as sv
        s["stat"] = sv.distill_loss(logits, s["token"], s["logprob"], temperature=c["temperature"],
                                    tail=c["tail"])["stat"]
    return s


def _prepare_prefix(c, g):
    N, W, page = c["N"], c["W"], c["page"]
    B = N * W
    plen = _ints(g, c["lo"], c["hi"], N)
    plen[-1] = c["hi"]
    lens = _ints(g, c["own_lo"], c["own_hi"], B)
    per_p, per = -(-c["hi"] // page), max(1, -(-c["own_hi"] // page))
    pool = N * per_p + B * per + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    ptable = order[:N * per_p].view(N, per_p)
    table = order[N * per_p:N * per_p + B * per].view(B, per)
    ptable = torch.where(torch.arange(per_p, device="cuda") * page < plen[:, None], ptable, -1)
    table = torch.where(torch.arange(per, device="cuda") * page < lens[:, None], table, -1)
    kv = torch.empty(2, pool, page, c["Hkv"], c["D"], dtype=_DT[c["dt"]], device="cuda")
    kv[0].normal_(generator=g)
    kv[1].normal_(generator=g)
    q = (_randn(g, B, c["Hq"], c["D"]) * 2).to(_DT[c["dt"]])
    s = dict(c=c, q=q, kv=kv, ptable=ptable.contiguous(), plen=plen, table=table.contiguous(),
             lens=lens)
    if own:
        import speculative_decoding_verification_vocab_gb300 as sv
        s["ws"] = torch.empty(sv.sv_prefix_attention_workspace(
            B, N, c["Hq"], c["Hkv"], c["D"], page, per_p, per), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"logprobs": _prepare_logprobs, "distill": _prepare_distill,
            "prefix": _prepare_prefix}[c["op"]](c, g)


# ------------------------------------------------------------- the plain forms
def _plain_logprobs(s):
    c, x, rows, tokens = s["c"], s["logits"], s["rows"], s["tokens"]
    P, V, K = c["P"], c["V"], c["K"]
    if rows is not None:
        x = x.gather(1, rows.clamp(min=0).long()[:, :, None].expand(-1, -1, V))
    x = x[:, :P].float()
    live = torch.ones(x.shape[:2], dtype=torch.bool, device=x.device) if tokens is None else tokens >= 0
    if rows is not None:
        live = live & (rows >= 0)
    m = x.amax(-1, keepdim=True)
    y = (x - m) / c["temperature"]
    e = torch.exp(y)
    l = e.sum(-1, keepdim=True)
    log_l = torch.log(l)
    r = dict(entropy=torch.where(live, (log_l - (e * y).sum(-1, keepdim=True) / l)[..., 0], 0.0))
    del e
    if tokens is not None:
        t = tokens.clamp(min=0).long()[..., None]
        r["logprob"] = torch.where(live, (y.gather(2, t) - log_l)[..., 0], 0.0)
    if K:
        # a number for each entry that orders by value, then by the lower index
        bits = (x + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() << 32
        key += V - 1 - torch.arange(V, device=x.device)
        top = key.topk(K, -1).values
        index = V - 1 - (top & 0xffffffff)
        r["top_token"] = torch.where(live[..., None], index, -1).to(torch.int32)
        r["top_logprob"] = torch.where(live[..., None], y.gather(2, index) - log_l, -math.inf)
    r["status"] = torch.zeros(x.shape[:2], dtype=torch.int32, device=x.device)
    return r


def _plain_distill(s):
    c, token, T = s["c"], s["token"].long(), s["c"]["temperature"]
    z = s["logits"].float() / T
    listed_z = z.gather(1, token)
    m = z.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    if c["tail"]:  # what the teacher's list leaves is one class more
        t = torch.exp(s["logprob"])
        t_rest = (1 - s["logprob"].double().exp().sum(1, keepdim=True)).clamp(min=0).float()
    else:
        t = torch.softmax(s["logprob"], 1)
        t_rest = torch.zeros_like(lse)
    rest = z.scatter(1, token, -math.inf)
    m_rest = rest.amax(1, keepdim=True)
    e_rest = torch.exp(rest - m_rest)
    l_rest = e_rest.sum(1, keepdim=True)
    lse_rest = m_rest + torch.log(l_rest)
    log_t = torch.log(torch.where(t > 0, t, 1.0))
    log_rest = torch.log(torch.where(t_rest > 0, t_rest, 1.0))
    r = {}
    if c["mode"] != "grad":
        loss = (t * (log_t - (listed_z - lse))).sum(1, keepdim=True)
        loss = loss + torch.where(t_rest > 0, t_rest * (log_rest - (lse_rest - lse)), 0.0)
        r["loss"] = loss[:, 0]
    if c["mode"] != "loss":
        w = 1.0 / T if s["weight"] is None else s["weight"][:, None] / T
        grad = e_rest * ((torch.exp(lse_rest - lse) - t_rest) / l_rest * w)
        grad = grad.scatter(1, token, (torch.exp(listed_z - lse) - t) * w)
        r["grad"] = s["grad"].copy_(grad)
    r["status"] = torch.zeros(c["R"], dtype=torch.int32, device=z.device)
    return r


def _plain_prefix(s):
    c, q, kv = s["c"], s["q"], s["kv"]
    N, W, Hkv, D, page = c["N"], c["W"], c["Hkv"], c["D"], c["page"]
    B = N * W

    def rows(table, lens):
        j = torch.arange(table.shape[1] * page, device=q.device)
        seen = j < lens[:, None]
        at = table.clamp(min=0).long()[:, j // page]
        k, v = (torch.where(seen[:, :, None, None], kv[i][at, j % page].float(), 0.0).transpose(1, 2)
                for i in range(2))
        return seen, k, v

    # [N][Hkv][W G][D] against the prefix, [B][Hkv][G][D] against a sequence's own slots
    x = q.float().view(N, W, Hkv, -1, D)
    G = x.shape[3]
    seen_p, k_p, v_p = rows(s["ptable"], s["plen"])
    seen_o, k_o, v_o = rows(s["table"], s["lens"])
    s_p = x.transpose(1, 2).reshape(N, Hkv, W * G, D) @ k_p.transpose(2, 3) * (D ** -0.5)
    s_p.masked_fill_(~seen_p[:, None, None], -math.inf)
    s_o = x.reshape(B, Hkv, G, D) @ k_o.transpose(2, 3) * (D ** -0.5)
    s_o.masked_fill_(~seen_o[:, None, None], -math.inf)

    def by_prefix(t):  # [B][Hkv][G][...] as [N][Hkv][W G][...]
        return t.view(N, W, Hkv, G, -1).transpose(1, 2).reshape(N, Hkv, W * G, -1)

    m = torch.maximum(s_p.amax(-1, keepdim=True), by_prefix(s_o.amax(-1, keepdim=True)))
    m_safe = torch.where(m == -math.inf, 0.0, m)
    e_p = s_p.sub_(m_safe).exp_()
    m_o = m_safe.view(N, Hkv, W, G, 1).transpose(1, 2).reshape(B, Hkv, G, 1)
    e_o = s_o.sub_(m_o).exp_()
    l = e_p.sum(-1, keepdim=True) + by_prefix(e_o.sum(-1, keepdim=True))
    out = (e_p @ v_p + by_prefix(e_o @ v_o)) / torch.where(l > 0, l, 1.0)
    lse = m + torch.log(l)

    def by_head(t):
        return t.view(N, Hkv, W, G, -1).transpose(1, 2).reshape(B, Hkv * G, -1)

    return dict(out=by_head(out).to(q.dtype), lse=by_head(lse)[..., 0],
                status=torch.zeros(B, dtype=torch.int32, device=q.device))


def run(state):
    s = state
    c = s["c"]
    op = c["op"]
    if not own:
        return {"logprobs": _plain_logprobs, "distill": _plain_distill, "prefix": _plain_prefix}[op](s)
    import speculative_decoding_verification_vocab_gb300 as sv
    if op == "logprobs":
        return sv.token_logprobs(s["logits"], s["tokens"], rows=s["rows"], top_k=c["K"],
                                 temperature=c["temperature"])
    if op == "distill":
        if c["mode"] == "grad":
            grad, status = sv.distill_grad(s["logits"], s["token"], s["logprob"], s["stat"],
                                           weight=s["weight"], temperature=c["temperature"],
                                           tail=c["tail"], out_grad=s["grad"])
            return dict(grad=grad, status=status)
        r = sv.distill_loss(s["logits"], s["token"], s["logprob"], weight=s["weight"],
                            temperature=c["temperature"], tail=c["tail"],
                            out_grad=s["grad"] if c["mode"] == "both" else None)
        return {k: r[k] for k in ("loss", "grad", "status") if k in r}
    out, lse, status = sv.prefix_attention(s["q"], s["kv"], s["ptable"], s["plen"], s["table"],
                                           s["lens"], return_lse=True, workspace=s["ws"])
    return dict(out=out, lse=lse, status=status)


# ---------------------------------------------------------------- floors, 64 bits
def work(case):
    c = dict(case)
    e = _BYTES[c["dt"]]
    if c["op"] == "logprobs":
        slots = c["B"] * c["P"]
        rows = slots if c["tokens"] in ("all", "none") else c["B"] * (1 + c["P"]) / 2
        ids = {"none": 0, "tree": 8}.get(c["tokens"], 4)
        outs = 8 + 8 * c["K"] + (0 if c["tokens"] == "none" else 4)
        return {"bytes": rows * c["V"] * e + slots * (ids + outs), "flops": rows * c["V"] * 5}
    if c["op"] == "distill":
        n = c["R"] * c["V"]
        grad = c["mode"] != "loss"
        return {"bytes": n * e * (2 if grad else 1) + c["R"] * (8 * c["K"] + 4 * c["weight"] + 8),
                "flops": n * ((4 if c["mode"] != "grad" else 0) + (4 if grad else 0))}
    B = c["N"] * c["W"]
    shared = c["N"] * (c["lo"] + c["hi"]) / 2
    own_slots = B * (c["own_lo"] + c["own_hi"]) / 2
    io = 2 * B * c["Hq"] * c["D"] * e + 4 * B * c["Hq"] + 4 * B
    table = 4 * (c["N"] + B + (shared + own_slots) / c["page"])
    return {"bytes": (shared + own_slots) * c["Hkv"] * 2 * c["D"] * e + io + table,
            "flops": 4 * c["D"] * c["Hq"] * (c["W"] * shared + own_slots)}


def _exact_logprobs(c, s):
    B, P, V, K = c["B"], c["P"], c["V"], c["K"]
    tokens, rows = s["tokens"], s["rows"]
    r = dict(entropy=torch.zeros(B, P, dtype=torch.float64, device="cuda"))
    if tokens is not None:
        r["logprob"] = torch.zeros(B, P, dtype=torch.float64, device="cuda")
    if K:
        r["top_logprob"] = torch.full((B, P, K), -math.inf, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // V)  # rows at a time
    live = torch.ones(B, P, dtype=torch.bool, device="cuda")
    if tokens is not None:
        live &= tokens >= 0
    at = live.nonzero()
    for i in range(0, len(at), step):
        b, p = at[i:i + step, 0], at[i:i + step, 1]
        x = s["logits"][b, p if rows is None else rows[b, p].long()].double() / c["temperature"]
        lp = x - torch.logsumexp(x, -1, keepdim=True)
        r["entropy"][b, p] = -torch.special.xlogy(lp.exp(), lp.exp()).sum(-1)
        if tokens is not None:
            r["logprob"][b, p] = lp.gather(1, tokens[b, p].long()[:, None])[:, 0]
        if K:
            r["top_logprob"][b, p] = lp.topk(K, -1).values
    return dict(r, top_token=None, status=None)


def _exact_distill(c, s):
    R, V = c["R"], c["V"]
    loss = torch.empty(R, dtype=torch.float64, device="cuda")
    grad = torch.empty(R, V, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 25) // V)
    for i in range(0, R, step):
        k = slice(i, i + step)
        log_s = torch.log_softmax(s["logits"][k].double() / c["temperature"], -1)
        idx, lt = s["token"][k].long(), s["logprob"][k].double()
        if not c["tail"]:
            lt = torch.log_softmax(lt, -1)
        t = lt.exp()
        loss[k] = (t * (lt - log_s.gather(1, idx))).sum(1)
        share = torch.ones(len(idx), 1, dtype=torch.float64, device="cuda")
        if c["tail"]:
            tr = (1 - t.sum(1)).clamp(min=0)
            lsr = torch.logsumexp(log_s.scatter(1, idx, -math.inf), 1)
            loss[k] += torch.special.xlogy(tr, tr) - tr * lsr
            share = 1 - (tr / lsr.exp())[:, None]
        else:
            share = share * t.sum(1, keepdim=True)
        probs = log_s.exp()
        g = (probs * share).scatter(1, idx, probs.gather(1, idx) - t) / c["temperature"]
        grad[k] = g if s["weight"] is None else g * s["weight"][k, None].double()
    r = dict(status=None)
    if c["mode"] != "grad":
        r["loss"] = loss
    if c["mode"] != "loss":
        r["grad"] = grad
    return r


def _exact_prefix(c, s):
    Hkv, D, page = c["Hkv"], c["D"], c["page"]
    outs, lses = [], []
    for b in range(c["N"] * c["W"]):
        parts = []
        for table, n in ((s["ptable"][b // c["W"]], int(s["plen"][b // c["W"]])),
                         (s["table"][b], int(s["lens"][b]))):
            j = torch.arange(n, device="cuda")
            parts.append(s["kv"][:, table[j // page].long(), j % page])
        k, v = torch.cat(parts, 1).double()
        x = torch.einsum("hgd,jhd->hgj", s["q"][b].double().view(Hkv, -1, D), k) / math.sqrt(D)
        lse = torch.logsumexp(x, -1)
        outs.append(torch.einsum("hgj,jhd->hgd", torch.exp(x - lse[..., None]), v).reshape(-1, D))
        lses.append(lse.reshape(-1))
    return dict(out=torch.stack(outs), lse=torch.stack(lses), status=None)


def exact(case, seed):
    """The outputs from their definitions in 64 bits, some rows or a sequence at a time."""
    c = dict(case)
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "distill": _exact_distill, "prefix": _exact_prefix}[c["op"]](c, s)
