"""Cases of the serving operators: page planning, appending keys and values to pages, and attention
over a shared prefix and paged caches.

``listed`` names the cases, ``draw`` gives more of the same ranges, ``prepare`` makes what a program
holds before a call, ``run`` makes one call, ``work`` counts what it cannot do without and ``exact``
computes the same outputs in 64 bits.  ``own`` selects the framework's operators; without it ``run``
computes the plain form: elementary torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

PAGE = 128


def listed():
    return [
        # page plan: a decode batch; a step that admits a few long prompts; a large ragged step
        dict(name="plan decode", op="plan", B=64, ctx_lo=1, ctx_hi=8000, new_lo=1, new_hi=1, pad=0),
        dict(name="plan prompts", op="plan", B=7, ctx_lo=0, ctx_hi=300, new_lo=500, new_hi=9000, pad=100),
        dict(name="plan ragged", op="plan", B=2000, ctx_lo=0, ctx_hi=5000, new_lo=0, new_hi=64, pad=1500),
        # append: one token per request of a decode batch; a batch of prompts; d = 64 with padded rows
        dict(name="append decode", op="append", N=64, Hkv=8, d=128, pad=0),
        dict(name="append prompts", op="append", N=16384, Hkv=8, d=128, pad=0),
        dict(name="append padded", op="append", N=1337, Hkv=12, d=64, pad=211),
        # attention: a single request answering a short prompt
        dict(name="attend one", op="attend", B=1, H=32, Hkv=8, d=128, prefix=256, own_lo=100, own_hi=100,
             new_lo=1, new_hi=1, pad=0),
        # a chat batch behind one system prompt
        dict(name="attend chat", op="attend", B=64, H=32, Hkv=8, d=128, prefix=4096, own_lo=1, own_hi=1024,
             new_lo=1, new_hi=1, pad=0),
        # many questions about one long document
        dict(name="attend document", op="attend", B=128, H=32, Hkv=8, d=128, prefix=32768, own_lo=20, own_hi=500,
             new_lo=1, new_hi=1, pad=0),
        # long conversations of their own, nothing shared
        dict(name="attend long", op="attend", B=32, H=32, Hkv=8, d=128, prefix=0, own_lo=1000, own_hi=32768,
             new_lo=1, new_hi=1, pad=0),
        # several drafted tokens per request to verify, one K/V head per query head, padded rows
        dict(name="attend drafts", op="attend", B=48, H=16, Hkv=16, d=64, prefix=1001, own_lo=9, own_hi=3001,
             new_lo=0, new_hi=8, pad=13),
        # a step that works prompt chunks beside decoding requests
        dict(name="attend chunks", op="attend", B=8, H=32, Hkv=4, d=128, prefix=2048, own_lo=1, own_hi=2300,
             new_lo=1, new_hi=600, pad=24),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend"])
    if op == "plan":
        B = _log(rng, 1, 2000)
        hi = min(9000, max(1, 60000 // B))
        new_hi = _log(rng, 1, hi)
        return dict(op=op, B=B, ctx_lo=rng.choice([0, 1, 127, 128]), ctx_hi=_log(rng, 128, 8000),
                    new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi, pad=rng.choice([0, 1, 100, 1000]))
    if op == "append":
        d, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8, 12, 16])
        return dict(op=op, N=_log(rng, 1, 16384 * 8 * 128 // (max(8, Hkv) * 128)), Hkv=Hkv, d=d,
                    pad=rng.choice([0, 0, 1, 77]))
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16] if d == 64 else [1, 2, 4, 8])
    H = Hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16) if Hkv * g <= 32])
    kind = rng.choice(["decode", "decode", "drafts", "chunks"])
    prefix = rng.choice([0, _log(rng, 1, 32768), _log(rng, 1, 32768)])
    if kind == "decode":
        B = _log(rng, 1, 128)
        own_hi = _log(rng, 1, min(32768, 500000 // B))
        return dict(op=op, B=B, H=H, Hkv=Hkv, d=d, prefix=prefix, own_lo=rng.randint(1, own_hi), own_hi=own_hi,
                    new_lo=1, new_hi=1, pad=rng.choice([0, 0, 3]))
    if kind == "drafts":
        B = _log(rng, 1, 48)
        own_hi = _log(rng, 16, 4000)
        return dict(op=op, B=B, H=H, Hkv=Hkv, d=d, prefix=min(prefix, 8192), own_lo=rng.randint(8, own_hi),
                    own_hi=own_hi, new_lo=rng.choice([0, 1, 4]), new_hi=rng.choice([4, 5, 8]), pad=rng.choice([0, 7]))
    own_hi = _log(rng, 700, 2300)
    return dict(op=op, B=_log(rng, 1, 8), H=H, Hkv=Hkv, d=d, prefix=min(prefix, 4096), own_lo=rng.randint(1, 600),
                own_hi=own_hi, new_lo=1, new_hi=_log(rng, 16, 600), pad=rng.choice([0, 24]))


def _spread(lo, hi, n):
    """n lengths evenly spaced from lo to hi (the upper one alone when n is 1)."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _lengths(case):
    """(own lengths with the new tokens, new tokens) of every request of an attention case, before they are put in
    an order: long and short chunks meet long and short caches, and a request has at least its new tokens."""
    B = case["B"]
    new = _spread(case["new_lo"], case["new_hi"], B)
    total = _spread(case["own_lo"], case["own_hi"], B)
    mixed = [total[(i * 5 + 3) % B] if math.gcd(5, B) == 1 else total[B - 1 - i] for i in range(B)]
    return [max(t, n) for t, n in zip(mixed, new)], new


def _ints(values, perm=None):
    t = torch.tensor(values, dtype=torch.int32)
    return (t if perm is None else t[perm]).cuda()


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device="cuda").manual_seed(seed)
    return dict(plan=_prepare_plan, append=_prepare_append, attend=_prepare_attend)[case["op"]](case, cpu, gpu)


def _prepare_plan(case, cpu, gpu):
    B = case["B"]
    ctx, new = _spread(case["ctx_lo"], case["ctx_hi"], B), _spread(case["new_lo"], case["new_hi"], B)
    perm, perm2 = torch.randperm(B, generator=cpu), torch.randperm(B, generator=cpu)
    ctx, new = torch.tensor(ctx)[perm], torch.tensor(new)[perm2]
    held = (ctx + PAGE - 1) // PAGE
    max_pages = _pages(case["ctx_hi"] + case["new_hi"]) + 1
    num_pages = int(held.sum()) + int(((new + PAGE - 1) // PAGE).sum()) + B + 5
    order = torch.randperm(num_pages, generator=cpu).to(torch.int32)
    first = torch.cumsum(held, 0) - held
    col = torch.arange(max_pages)
    table = torch.where(col < held[:, None], order[(first[:, None] + col).clamp(max=num_pages - 1)], -1)
    max_tokens = int(new.sum()) + case["pad"]
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(op="plan", ctx=ctx.to(torch.int32).cuda(), new=new.to(torch.int32).cuda(),
                free=order[int(held.sum()):].contiguous().cuda(), head=torch.full((1,), 3, **i32),
                table=table.to(torch.int32).contiguous().cuda(), num_pages=num_pages, max_tokens=max_tokens,
                seq=torch.empty(B, **i32), cu=torch.empty(B + 1, **i32), slots=torch.empty(max(1, max_tokens), **i32),
                head_out=torch.empty(1, **i32))


def _prepare_append(case, cpu, gpu):
    N, Hkv, d, pad = case["N"], case["Hkv"], case["d"], case["pad"]
    num_pages = _pages(N) + 3
    slots = torch.randperm(num_pages * PAGE, generator=cpu)[:N + pad].to(torch.int32)
    if N >= PAGE:  # prompts: runs of tokens in pages; the last rows of the batch hold no token
        pages = torch.randperm(num_pages, generator=cpu)[:_pages(N)]
        slots[:N] = ((pages[:, None] * PAGE + torch.arange(PAGE)).reshape(-1)[:N]).to(torch.int32)
    slots[N:] = -1
    # the new keys and values are columns of one projection's output, as a model produces them
    kv = torch.randn(N + pad, 2 * Hkv * d, generator=gpu, device="cuda").to(torch.bfloat16)
    k_new, v_new = kv[:, :Hkv * d].unflatten(1, (Hkv, d)), kv[:, Hkv * d:].unflatten(1, (Hkv, d))
    # one page more than the operators are told of: the plain form puts padded rows there
    store = torch.randn(2, num_pages + 1, Hkv, PAGE, d, generator=gpu, device="cuda", dtype=torch.bfloat16)
    return dict(op="append", k_new=k_new, v_new=v_new, slots=slots.cuda(), k_store=store[0], v_store=store[1],
                k_pages=store[0, :num_pages], v_pages=store[1, :num_pages], num_pages=num_pages)


def _prepare_attend(case, cpu, gpu):
    B, H, Hkv, d, P = case["B"], case["H"], case["Hkv"], case["d"], case["prefix"]
    total, new = _lengths(case)
    perm = torch.randperm(B, generator=cpu)
    total, new = torch.tensor(total)[perm], torch.tensor(new)[perm]
    held = (total + PAGE - 1) // PAGE
    max_pages = max(1, int(held.max()))
    num_pages = _pages(P) + int(held.sum()) + 1
    order = torch.randperm(num_pages, generator=cpu).to(torch.int32)
    first = _pages(P) + torch.cumsum(held, 0) - held
    col = torch.arange(max_pages)
    table = torch.where(col < held[:, None], order[(first[:, None] + col).clamp(max=num_pages - 1)], -1)
    rows = int(new.sum()) + case["pad"]
    pool = torch.randn(2, num_pages, Hkv, PAGE, d, generator=gpu, device="cuda", dtype=torch.bfloat16)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(new, 0)])
    state = dict(op="attend", q=torch.randn(rows, H, d, generator=gpu, device="cuda").to(torch.bfloat16),
                 k_pages=pool[0], v_pages=pool[1], prefix_len=P, max_new=case["new_hi"], scale=d ** -0.5,
                 prefix_table=order[:max(1, _pages(P))].contiguous().cuda(),
                 table=table.to(torch.int32).contiguous().cuda(), seq=total.to(torch.int32).cuda(),
                 cu=cu.to(torch.int32).cuda(), o=torch.zeros(rows, H, d, dtype=torch.bfloat16, device="cuda"),
                 lse=torch.zeros(rows, H, device="cuda"), workspace=None)
    if own:
        import exact_io_aware_07_gb300 as fa

        state["workspace"] = torch.empty(fa.fa_fwd_prefix_paged_workspace_bytes(rows, B, H, Hkv, d),
                                         dtype=torch.uint8, device="cuda")
    return state


def run(state):
    if own:
        return _run_own(state)
    return dict(plan=_plan, append=_append, attend=_attend)[state["op"]](state)


def _run_own(s):
    import exact_io_aware_07_gb300 as fa

    if s["op"] == "plan":
        fa.fa_page_plan(s["ctx"], s["new"], s["free"], s["head"], s["table"], s["seq"], s["cu"], s["slots"],
                        s["head_out"], s["num_pages"])
        return s["table"], s["seq"], s["cu"], s["slots"], s["head_out"]
    if s["op"] == "append":
        fa.fa_kv_append(s["k_new"], s["v_new"], s["slots"], s["k_pages"], s["v_pages"])
        return s["k_pages"], s["v_pages"]
    fa.fa_fwd_prefix_paged(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], s["prefix_len"], s["table"],
                           s["seq"], s["cu"], s["max_new"], s["o"], s["lse"], True, s["scale"], s["workspace"])
    return s["o"], s["lse"]


def _plan(s):
    ctx, new, dev = s["ctx"].long(), s["new"].long(), s["ctx"].device
    seq = ctx + new
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(new, 0)])
    p0, p1 = (ctx + PAGE - 1) // PAGE, (seq + PAGE - 1) // PAGE
    taken = torch.cumsum(p1 - p0, 0)
    first = s["head"].long() + taken - (p1 - p0)
    col = torch.arange(s["table"].shape[1], device=dev)
    fresh = (col >= p0[:, None]) & (col < p1[:, None])
    index = (first[:, None] + col - p0[:, None]).clamp(0, max(0, s["free"].numel() - 1))
    if s["free"].numel():
        s["table"].copy_(torch.where(fresh, s["free"][index], s["table"]))
    t = torch.arange(s["slots"].numel(), device=dev)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=ctx.numel() - 1)
    pos = (ctx[b] + t - cu[b]).clamp(max=s["table"].shape[1] * PAGE - 1)
    slot = s["table"][b, pos // PAGE].long() * PAGE + pos % PAGE
    s["slots"].copy_(torch.where(t < cu[-1], slot, -1))
    s["seq"].copy_(seq)
    s["cu"].copy_(cu)
    s["head_out"].copy_(s["head"] + taken[-1])
    return s["table"], s["seq"], s["cu"], s["slots"], s["head_out"]


def _append(s):
    slot = s["slots"].long()
    slot = torch.where(slot >= 0, slot, s["num_pages"] * PAGE)
    s["k_store"][slot // PAGE, :, slot % PAGE] = s["k_new"]
    s["v_store"][slot // PAGE, :, slot % PAGE] = s["v_new"]
    return s["k_pages"], s["v_pages"]


def _attend(s):
    q, cu, seq = s["q"].float(), s["cu"].long(), s["seq"].long()
    N, H, d = q.shape
    Hkv, group, T = s["k_pages"].shape[1], H // s["k_pages"].shape[1], s["max_new"]
    B, dev = seq.numel(), q.device
    # the prefix, for all rows at once: (Hkv, N * group, P)
    P = s["prefix_len"]
    pages = s["prefix_table"][:_pages(P)].long()
    kp = s["k_pages"][pages].float().transpose(0, 1).reshape(Hkv, -1, d)[:, :P]
    vp = s["v_pages"][pages].float().transpose(0, 1).reshape(Hkv, -1, d)[:, :P]
    qg = q.view(N, Hkv, group, d)
    sp = s["scale"] * (qg.transpose(0, 1).reshape(Hkv, N * group, d) @ kp.transpose(1, 2))
    sp = sp.view(Hkv, N, group, P)
    # own keys, request by request in a padded batch: (B, Hkv, T * group, L)
    table = s["table"].long().clamp(min=0)
    L = table.shape[1] * PAGE
    ko = s["k_pages"][table].float().transpose(1, 2).reshape(B, Hkv, L, d)
    vo = s["v_pages"][table].float().transpose(1, 2).reshape(B, Hkv, L, d)
    n = torch.arange(N, device=dev)
    b = torch.searchsorted(cu[1:], n, right=True).clamp(max=B - 1)
    i = (n - cu[b]).clamp(max=T - 1)
    tok = (cu[:-1, None] + torch.arange(T, device=dev)).clamp(max=max(0, N - 1))
    qo = qg[tok].permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * group, d)
    so = s["scale"] * (qo @ ko.transpose(2, 3)).view(B, Hkv, T, group, L)
    last = (seq - (cu[1:] - cu[:-1]))[:, None] + torch.arange(T, device=dev)  # the last own key a token sees
    seen = torch.arange(L, device=dev) <= torch.minimum(last, seq[:, None] - 1)[:, :, None]
    so = torch.where(seen[:, None, :, None, :], so, -math.inf)
    m = so.amax(-1)[b, :, i]  # (N, Hkv, group)
    if P:
        m = torch.maximum(m, sp.amax(-1).transpose(0, 1))
    m = torch.where(m == -math.inf, 0.0, m)
    live = (n < cu[-1])[:, None, None]
    mo = torch.zeros(B + 1, T, Hkv, group, device=dev)  # the last one takes the rows behind the last request
    mo[torch.where(n < cu[-1], b, B), i] = m
    wo = torch.exp(so - mo[:B].permute(0, 2, 1, 3)[..., None])
    acc = (wo.reshape(B, Hkv, T * group, L) @ vo).view(B, Hkv, T, group, d)[b, :, i]
    total = wo.sum(-1)[b, :, i]
    if P:
        wp = torch.exp(sp - m.transpose(0, 1)[..., None])
        acc = acc + (wp.view(Hkv, N * group, P) @ vp).view(Hkv, N, group, d).transpose(0, 1)
        total = total + wp.sum(-1).transpose(0, 1)
    o = acc / torch.where(total > 0, total, 1.0)[..., None]
    lse = m + torch.log(total)
    s["o"].copy_(torch.where(live, o.reshape(N, H, d).to(torch.bfloat16), s["o"]))
    s["lse"].copy_(torch.where(live[..., 0], lse.reshape(N, H), s["lse"]))
    return s["o"], s["lse"]


def work(case):
    if case["op"] == "plan":
        B = case["B"]
        new = _spread(case["new_lo"], case["new_hi"], B)
        # the lengths meet in an order of the seed's: new pages on average
        fresh = sum(new) // PAGE + B // 2
        return dict(bytes=20 * B + 8 * fresh + 4 * (sum(new) + case["pad"]), flops=0)
    if case["op"] == "append":
        row = case["Hkv"] * case["d"] * 2
        return dict(bytes=4 * (case["N"] + case["pad"]) + 4 * case["N"] * row, flops=0)
    H, Hkv, d, P = case["H"], case["Hkv"], case["d"], case["prefix"]
    total, new = _lengths(case)
    rows = sum(new)
    keys = P + sum(t for t, n in zip(total, new) if n)
    seen = rows * P + sum(n * t - n * (n - 1) // 2 for t, n in zip(total, new))
    return dict(bytes=keys * Hkv * d * 4 + rows * H * (4 * d + 4), flops=4 * d * H * seen)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "plan":
        return _exact_plan(s)
    if s["op"] == "append":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        for x, pages in ((s["k_new"], k), (s["v_new"], v)):
            rows = pages.permute(0, 2, 1, 3).reshape(-1, pages.shape[1], pages.shape[3])
            held = [(t, w) for t, w in enumerate(s["slots"].tolist()) if w >= 0]
            rows[[w for _, w in held]] = x[[t for t, _ in held]].double()
            pages.copy_(rows.view(pages.shape[0], PAGE, pages.shape[1], pages.shape[3]).permute(0, 2, 1, 3))
        return k, v
    return _exact_attend(s)


def _exact_plan(s):
    ctx, new, free = s["ctx"].tolist(), s["new"].tolist(), s["free"].tolist()
    table, head = s["table"].tolist(), int(s["head"])
    cu, slots = [0], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        for t in range(c, c + n):
            if t % PAGE == 0:
                table[b][t // PAGE] = free[head]
                head += 1
            slots.append(table[b][t // PAGE] * PAGE + t % PAGE)
        cu.append(cu[-1] + n)
    slots += [-1] * (s["slots"].numel() - len(slots))
    return tuple(torch.tensor(x, dtype=torch.int32)
                 for x in (table, [c + n for c, n in zip(ctx, new)], cu, slots, [head]))


def _exact_attend(s):
    cu, seq = s["cu"].tolist(), s["seq"].tolist()
    N, H, d = s["q"].shape
    Hkv = s["k_pages"].shape[1]
    group = H // Hkv
    o = torch.zeros(N, H, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(N, H, dtype=torch.float64, device="cuda")
    P = s["prefix_len"]

    def keys(pages, table, n):
        return pages[table[:_pages(n)].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].double()

    kp, vp = (keys(x, s["prefix_table"], P) for x in (s["k_pages"], s["v_pages"]))
    for b, n in enumerate(seq):
        rows = cu[b + 1] - cu[b]
        if rows == 0:
            continue
        ko, vo = (keys(x, s["table"][b], n) for x in (s["k_pages"], s["v_pages"]))
        q = s["q"][cu[b]:cu[b + 1]].double().view(rows, Hkv, group, d)
        past = torch.arange(n, device="cuda") > (n - rows + torch.arange(rows, device="cuda"))[:, None]
        for g in range(Hkv):
            own_scores = torch.einsum("thd,kd->thk", q[:, g], ko[g]).masked_fill(past[:, None], -math.inf)
            x = s["scale"] * torch.cat([torch.einsum("thd,kd->thk", q[:, g], kp[g]), own_scores], -1)
            z = torch.logsumexp(x, -1)
            w = torch.exp(x - z[..., None])
            at = slice(cu[b], cu[b + 1]), slice(g * group, (g + 1) * group)
            o[at] = torch.einsum("thk,kd->thd", w[..., :P], vp[g]) + torch.einsum("thk,kd->thd", w[..., P:], vo[g])
            lse[at] = z
    return o, lse
