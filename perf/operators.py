"""The serving operators beside verification -- decode attention over a paged
KV cache, eviction from it by accumulated attention weight, and verification
of drafted tokens from probabilities and given random numbers -- as measured
cases: their inputs, their plain form, the framework's calls and a 64-bit
form.

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
        # a draft model's step for one user: short context, latency counts
        dict(name="attn_one_short", op="attn", B=1, Hq=32, Hkv=8, D=128, lo=200, hi=213, page=16,
             dt="bf16", window=0, sinks=0, weights=False),
        # the dynamic-tree workload's layer (64 query heads on 8 KV heads of
        # 128, about 4096 tokens of context, 128 sequences) decoding
        dict(name="attn_batch", op="attn", B=128, Hq=64, Hkv=8, D=128, lo=3585, hi=4096, page=16,
             dt="bf16", window=0, sinks=0, weights=False),
        # one long document: the work has to be split over the cache's length
        dict(name="attn_one_long", op="attn", B=1, Hq=64, Hkv=8, D=128, lo=131001, hi=131001,
             page=64, dt="bf16", window=0, sinks=0, weights=False),
        # a draft model that streams: a window and a few first tokens, one
        # query head per KV head, small heads, fp16
        dict(name="attn_window", op="attn", B=64, Hq=16, Hkv=16, D=64, lo=1500, hi=20000, page=32,
             dt="f16", window=2048, sinks=4, weights=False),
        # a cache under a budget: the weights each slot receives are summed
        dict(name="attn_weights", op="attn", B=24, Hq=32, Hkv=4, D=128, lo=1000, hi=8500, page=20,
             dt="bf16", window=0, sinks=0, weights=True),
        # one sequence, one layer, a little over its budget
        dict(name="evict_one", op="evict", L=1, B=1, Hkv=8, D=128, lo=1101, hi=1101, page=16,
             dt="bf16", budget=1024, sinks=4, recent=256),
        # several layers of a batch, back to half of their length
        dict(name="evict_batch", op="evict", L=8, B=32, Hkv=8, D=128, lo=1900, hi=2300, page=16,
             dt="bf16", budget=1024, sinks=4, recent=128),
        # one long document cut to a quarter
        dict(name="evict_one_long", op="evict", L=2, B=1, Hkv=8, D=128, lo=131001, hi=131001,
             page=64, dt="bf16", budget=32768, sinks=16, recent=4096),
        # the tiny chain: one user, small vocabulary, latency
        dict(name="verify_tiny", op="verify", B=1, N=4, V=1000, dt="f32", drafts="probs", pad=0,
             ragged=False),
        # the batched chain's shape, probabilities rounded to bf16
        dict(name="verify_batch", op="verify", B=64, N=5, V=32000, dt="bf16", drafts="probs",
             pad=0, ragged=True),
        # the large-vocabulary chain
        dict(name="verify_large", op="verify", B=256, N=7, V=128256, dt="f32", drafts="probs",
             pad=0, ragged=False),
        # drafts copied from the prompt (no draft distribution), odd vocabulary
        # in rows padded to a multiple of 64
        dict(name="verify_onehot", op="verify", B=96, N=7, V=40001, dt="f32", drafts="onehot",
             pad=63, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "evict", "verify", "verify"])
    if op == "attn":
        Hkv = rng.choice([1, 2, 4, 8, 16])
        G = rng.choice([1, 2, 3, 4, 7, 8, 16])
        D = rng.choice([64, 128, 128, 256])
        B = _log_int(rng, 1, 128)
        hi = _log_int(rng, 17, max(18, min(131072, 1900000000 // (B * Hkv * D * 4))))
        window = _log_int(rng, 16, 4096) if rng.random() < 0.35 else 0
        return dict(op="attn", B=B, Hq=Hkv * G, Hkv=Hkv, D=D, lo=max(1, hi // rng.choice([1, 2, 8])),
                    hi=hi, page=rng.choice([1, 8, 16, 24, 32, 64, 128]), dt=rng.choice(["bf16", "f16"]),
                    window=window, sinks=rng.choice([0, 1, 4, 33]) if window else 0,
                    weights=rng.random() < 0.3)
    if op == "evict":
        Hkv = rng.choice([1, 2, 4, 8])
        D = rng.choice([64, 128, 256])
        L = rng.choice([1, 1, 2, 5])
        B = _log_int(rng, 1, 32)
        hi = _log_int(rng, 64, max(65, min(131072, (1 << 29) // (L * B * Hkv * D * 4))))
        budget = max(16, int(hi * rng.choice([0.3, 0.5, 0.9])))
        sinks = rng.choice([0, 1, 4])
        return dict(op="evict", L=L, B=B, Hkv=Hkv, D=D, lo=max(1, hi // rng.choice([1, 2])), hi=hi,
                    page=rng.choice([8, 16, 24, 64]), dt=rng.choice(["bf16", "f16", "f32"]),
                    budget=budget, sinks=sinks,
                    recent=rng.choice([0, 1, max(1, budget // 4), budget - sinks]))
    V = _log_int(rng, 17, 128256)
    N = rng.choice([1, 2, 3, 5, 7, 12])
    dt = rng.choice(["f32", "f32", "bf16"])
    B = _log_int(rng, 1, max(2, min(512, (1 << 29) // ((2 * N + 1) * V))))
    return dict(op="verify", B=B, N=N, V=V, dt=dt, drafts=rng.choice(["probs", "probs", "onehot"]),
                pad=rng.choice([0, 0, 7, 64]), ragged=rng.random() < 0.5)


# ----------------------------------------------------------------- the inputs
def _pages(c, g, layers):
    """Lengths, a page table in random order (-1 where a sequence needs no
    page) and a page pool [layers][2][pages][page][Hkv][D] with some spare."""
    B, page = c["B"], c["page"]
    lens = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g, device="cuda")
    lens[torch.randint(0, B, (1,), generator=g, device="cuda")] = c["hi"]
    per = -(-c["hi"] // page)
    pool = B * per + max(3, B * per // 32)
    table = torch.randperm(pool, generator=g, device="cuda")[:B * per].view(B, per)
    used = torch.arange(per, device="cuda") * page < lens[:, None]
    if c.get("window"):  # pages behind the window have been given back
        end = (torch.arange(per, device="cuda") + 1) * page
        start = torch.arange(per, device="cuda") * page
        used &= (end > (lens - c["window"])[:, None]) | (start < c["sinks"])
    table = torch.where(used, table, -1).to(torch.int32)
    shape = (2, pool, page, c["Hkv"], c["D"])
    kv = torch.empty((layers,) + shape, dtype=_DT[c["dt"]], device="cuda")
    for i in range(layers):
        for j in range(2):
            kv[i, j].normal_(generator=g)
    return lens.to(torch.int32), table.contiguous(), kv


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if c["op"] == "attn":
        lens, table, kv = _pages(c, g, 1)
        # scores of a few units' spread, as trained heads have them
        q = (torch.randn(c["B"], c["Hq"], c["D"], generator=g, device="cuda") * 2).to(_DT[c["dt"]])
        s = dict(c=c, q=q, kv=kv[0], table=table, lens=lens, sums=None)
        if c["weights"]:
            s["sums"] = torch.rand(c["B"], c["Hkv"], table.shape[1] * c["page"], generator=g,
                                   device="cuda")
        if own:
            import speculative_decoding_verification_vocab_gb300 as sv
            s["ws"] = torch.empty(sv.sv_paged_attention_workspace(
                c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], table.shape[1], c["window"],
                c["sinks"], c["weights"]), dtype=torch.uint8, device="cuda")
        return s
    if c["op"] == "evict":
        lens, table, kv = _pages(c, g, c["L"])
        S = table.shape[1] * c["page"]
        # heavy-tailed sums, a tenth of the slots never attended to (ties at 0)
        w = torch.randn(c["L"], c["B"], c["Hkv"], S, generator=g, device="cuda").mul_(1.5).exp_()
        w *= torch.rand(w.shape, generator=g, device="cuda") > 0.1
        w *= torch.arange(S, device="cuda") < lens[:, None, None]
        s = dict(c=c, kv=kv, table=table, lens=lens, sums=w, out_sums=torch.zeros_like(w))
        if own:
            import speculative_decoding_verification_vocab_gb300 as sv
            s["ws"] = torch.empty(sv.sv_kv_evict_workspace(c["L"], c["B"], c["Hkv"], c["budget"]),
                                  dtype=torch.uint8, device="cuda")
        return s
    B, N, V = c["B"], c["N"], c["V"]
    ld = V + c["pad"]
    dt = _DT[c["dt"]]
    q = torch.zeros(B, N + 1, ld, dtype=dt, device="cuda")
    p = torch.zeros(B, N, ld, dtype=dt, device="cuda") if c["drafts"] == "probs" else None
    d = torch.empty(B, N, dtype=torch.int32, device="cuda")
    for i in range(N + 1):  # a draft that tracks the target: most tokens are accepted
        x = torch.randn(B, V, generator=g, device="cuda") * 3
        q[:, i, :V] = torch.softmax(x, -1).to(dt)
        if i < N:
            y = x + 0.3 * torch.randn(B, V, generator=g, device="cuda")
            if p is not None:
                p[:, i, :V] = torch.softmax(y, -1).to(dt)
            noise = torch.rand(B, V, generator=g, device="cuda").clamp_(1e-20, 1 - 1e-7)
            if p is None:  # a copied token is right more often than a drawn one
                y = x * 2
            d[:, i] = (y - torch.log(-torch.log(noise))).argmax(-1)
    u = torch.rand(B, N, generator=g, device="cuda")
    us = torch.rand(B, generator=g, device="cuda")
    if p is None:
        u *= 0.2
    n = torch.randint(0, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if c["ragged"] else None
    return dict(c=c, q=q[:, :, :V], p=None if p is None else p[:, :, :V], d=d, u=u, us=us, n=n)


# ------------------------------------------------------------- the plain forms
def _plain_attention(s):
    c, q, kv, table, lens = s["c"], s["q"], s["kv"], s["table"], s["lens"].long()
    B, Hkv, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    cap = table.shape[1] * page
    # the visible slots of each sequence, in order: the first tokens, then the window
    lo = (lens - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    first = lo.clamp(max=c["sinks"])
    width = min(cap, c["sinks"] + c["window"]) if c["window"] else cap
    i = torch.arange(width, device=q.device)
    slot = torch.where(i < first[:, None], i, i - first[:, None] + lo[:, None])
    seen = slot < lens[:, None]
    slot = torch.where(seen, slot, 0)
    row = table.gather(1, slot // page).clamp(min=0).long()
    mask = seen[:, None, :, None]
    k = torch.where(mask, kv[0][row, slot % page].transpose(1, 2).float(), 0.0)
    v = torch.where(mask, kv[1][row, slot % page].transpose(1, 2).float(), 0.0)
    x = q.float().view(B, Hkv, -1, D) @ k.transpose(2, 3) * (D ** -0.5)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = e.sum(-1, keepdim=True)
    w = e / torch.where(l > 0, l, 1.0)
    out = (w @ v).view(q.shape).to(q.dtype)
    lse = (m + torch.log(l)).view(B, -1)
    r = dict(out=out, lse=lse)
    if s["sums"] is not None:
        s["sums"].scatter_add_(2, slot[:, None].expand(B, Hkv, width),
                               torch.where(seen[:, None], w.sum(2), 0.0))
        r["weight_sum"] = s["sums"]
    return r


def _plain_evict(s):
    c, kv, table, lens = s["c"], s["kv"], s["table"], s["lens"].long()
    L, B, H, page, m = c["L"], c["B"], c["Hkv"], c["page"], c["budget"]
    w = s["sums"]
    S = w.shape[3]
    m = min(m, S)
    j = torch.arange(S, device=w.device)
    n = lens[:, None, None]
    # what is kept without question stands above every weight, what is past the end below
    key = torch.where((j < c["sinks"]) | (j >= n - c["recent"]), math.inf, w)
    key = torch.where(j < n, key, -math.inf)
    kept = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :m].sort(-1).values
    kept = torch.where(n > m, kept, j[:m])
    has = j[:m] < n
    src = torch.where(has, kept, 0)
    rows = torch.gather(w, 3, src)
    out_w = s["out_sums"]
    new = torch.nn.functional.pad(torch.where(has, rows, 0.0), (0, S - m))
    out_w.copy_(torch.where(j < n, new, out_w))
    # rows of the page pool, K and V, of every layer at once
    t = table.clamp(min=0).long()
    bi = torch.arange(B, device=w.device)[:, None, None]
    hi = torch.arange(H, device=w.device)[:, None]
    li = torch.arange(L, device=w.device)[:, None, None, None]
    move = kept != j[:m]
    at = move.nonzero(as_tuple=True)
    frm, to = kept[at], at[3]
    l_, b_, h_ = at[0], at[1], at[2]
    vals = kv[l_, :, t[b_, frm // page], frm % page, h_]
    kv[l_, :, t[b_, to // page], to % page, h_] = vals
    return dict(kept=torch.where(has, kept, -1).to(torch.int32), kv_len=lens.clamp(max=m).to(torch.int32),
                weight_sum=out_w, kv=kv)


def _plain_verify(s):
    q, p, d, u, us, n = s["q"], s["p"], s["d"].long(), s["u"], s["us"], s["n"]
    B, N = d.shape
    if n is None:
        n = torch.full((B,), N, device=d.device)
    n = n.long()
    qd = q[:, :N].gather(2, d[..., None])[..., 0].double()
    pd = p.gather(2, d[..., None])[..., 0].double() if p is not None else torch.ones_like(qd)
    ok = ((u.double() * pd < qd) | (pd == 0)) & (torch.arange(N, device=d.device) < n[:, None])
    a = ok.long().cumprod(1).sum(1)
    b = torch.arange(B, device=d.device)
    qa = q[b, a].float()
    at = a.clamp(max=N - 1)
    if p is not None:
        pa = p[b, at].float()
    else:
        pa = torch.zeros_like(qa)
        pa[b, d[b, at]] = 1.0
    rejected = (a < n)[:, None]
    w = torch.where(rejected, (qa - pa).clamp(min=0), qa)
    none = w.sum(1, keepdim=True) == 0
    w = torch.where(none, qa, w)
    cum = w.double().cumsum(1)
    token = (cum <= us.double()[:, None] * cum[:, -1:]).sum(1)
    i = torch.arange(N + 1, device=d.device)
    drafts = torch.nn.functional.pad(d, (0, 1))
    tokens = torch.where(i < a[:, None], drafts, torch.where(i == a[:, None], token[:, None], -1))
    status = 4 * (none[:, 0] & rejected[:, 0]).int() + 8 * ((pd == 0) & (torch.arange(N, device=d.device) < a[:, None])).any(1).int()
    return dict(tokens=tokens.to(torch.int32), accept_len=a.to(torch.int32), status=status)


def run(state):
    s = state
    op = s["c"]["op"]
    if not own:
        return {"attn": _plain_attention, "evict": _plain_evict, "verify": _plain_verify}[op](s)
    import speculative_decoding_verification_vocab_gb300 as sv
    c = s["c"]
    if op == "attn":
        out, lse, _ = sv.paged_attention(s["q"], s["kv"], s["table"], s["lens"], window=c["window"],
                                         sinks=c["sinks"], weight_sum=s["sums"], return_lse=True,
                                         workspace=s["ws"])
        r = dict(out=out, lse=lse)
        if s["sums"] is not None:
            r["weight_sum"] = s["sums"]
        return r
    if op == "evict":
        kept, kv_len, _ = sv.kv_evict(s["kv"], s["table"], s["lens"], s["sums"], c["budget"],
                                      sinks=c["sinks"], recent=c["recent"],
                                      out_weight_sum=s["out_sums"], workspace=s["ws"])
        return dict(kept=kept, kv_len=kv_len, weight_sum=s["out_sums"], kv=s["kv"])
    r = sv.verify_chain_probs(s["q"], s["p"], s["d"], s["u"], s["us"], n_draft=s["n"])
    return dict(tokens=r["tokens"], accept_len=r["accept_len"], status=r["status"])


# ---------------------------------------------------------------- floors, 64 bits
def work(case):
    c = dict(case)
    mean = (c["lo"] + c["hi"]) / 2 if "lo" in c else 0
    if c["op"] == "attn":
        e = _BYTES[c["dt"]]
        seen = min(mean, c["window"] + c["sinks"]) if c["window"] else mean
        slots = c["B"] * c["Hkv"] * seen
        io = 2 * c["B"] * c["Hq"] * c["D"] * e + 4 * c["B"] * c["Hq"]
        table = 4 * c["B"] * (1 + seen / c["page"])
        return {"bytes": slots * 2 * c["D"] * e + io + table + (8 * slots if c["weights"] else 0),
                "flops": 4 * c["D"] * c["Hq"] / c["Hkv"] * slots}
    if c["op"] == "evict":
        e = _BYTES[c["dt"]]
        n, m = mean, min(c["budget"], mean)
        heads = c["L"] * c["B"] * c["Hkv"]
        # the first tokens stay where they are; every other kept row is read and written
        moved = (m - c["sinks"]) if n > m else 0
        return {"bytes": heads * (moved * 2 * c["D"] * e * 2 + 8 * n + 4 * m) + 4 * c["B"] * n / c["page"],
                "flops": heads * n}
    e = _BYTES[c["dt"]]
    rows = 2 if c["drafts"] == "probs" else 1
    return {"bytes": c["B"] * (rows * c["V"] * e + c["N"] * (8 + rows * e) + 4 * (c["N"] + 3)),
            "flops": c["B"] * 2 * c["V"]}


def exact(case, seed):
    """The outputs from their definitions in 64 bits, sequence by sequence."""
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] == "verify":
        return None  # whole numbers only
    page = c["page"]
    if c["op"] == "evict":
        w = s["sums"].cpu().double()
        out = s["out_sums"].cpu().double()
        L, B, H, S = w.shape
        for b in range(B):
            n = int(s["lens"][b])
            m = min(c["budget"], n)
            for l in range(L):
                for h in range(H):
                    x = w[l, b, h, :n].numpy()
                    if n > c["budget"]:
                        mid = sorted(range(c["sinks"], n - c["recent"]), key=lambda j: (-x[j], j))
                        mid = mid[:m - c["sinks"] - c["recent"]] if m > c["sinks"] + c["recent"] else []
                        keep = list(range(c["sinks"])) + sorted(mid) + list(range(n - c["recent"], n))
                    else:
                        keep = list(range(n))
                    out[l, b, h, :n] = 0
                    out[l, b, h, :m] = w[l, b, h, keep]
        return dict(kept=None, kv_len=None, weight_sum=out, kv=None)
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    outs, lses = [], []
    sums = s["sums"].double() if s["sums"] is not None else None
    for b in range(B):
        n = int(s["lens"][b])
        j = torch.arange(n, device="cuda")
        if c["window"]:
            j = j[(j >= n - c["window"]) | (j < c["sinks"])]
        pages = s["table"][b, j // page].long()
        k = s["kv"][0, pages, j % page].double()
        v = s["kv"][1, pages, j % page].double()
        qb = s["q"][b].double().view(Hkv, G, D)
        x = torch.einsum("hgd,jhd->hgj", qb, k) / math.sqrt(D)
        lse = torch.logsumexp(x, -1)
        a = torch.exp(x - lse[..., None])
        outs.append(torch.einsum("hgj,jhd->hgd", a, v).reshape(Hq, D))
        lses.append(lse.reshape(Hq))
        if sums is not None:
            sums[b][:, j] += a.sum(1)
    r = dict(out=torch.stack(outs), lse=torch.stack(lses))
    if sums is not None:
        r["weight_sum"] = sums
    return r
