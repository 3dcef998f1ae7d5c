"""The serving operators of Stochastic Attention, measured: a paged K/V cache, what fills it and the
attention that reads it.

- plan:   block tables, token slots and positions of a ragged batch, from its requests' lengths
- append: rotated keys and values of the new tokens into the pages (and the queries rotated)
- swa:    sliding-window (or full causal) attention of the new tokens over the cache
- sa:     causal Stochastic Attention of the new tokens over the cache
- gated:  the sigmoid-gated sum of the two

A request's new tokens are its last ones: with L tokens in all, n of them new, new token i has
position L - n + i.  Position p of a request lives in row p % page of page block_table[b, p // page].
"""

import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    gqa = dict(hq=32, hkv=8, d=128)  # the long-prefill shape of the benchmark
    return [
        # one user, one token, a short conversation: nothing but latency
        dict(name="swa_one_token", op="swa", batch=1, new=1, kind="decode", ctx=1000, window=128, page=16, **gqa),
        # a decoding batch with full attention over long ragged contexts: the cache read is everything
        dict(name="swa_decode_long", op="swa", batch=48, new=1, kind="decode", ctx=32768, window=1 << 20, page=64, **gqa),
        # a chunk of a long prompt over its cached first part, full attention: matrix products
        dict(name="swa_chunk_full", op="swa", batch=1, new=2048, kind="chunk", ctx=32768, window=1 << 20, page=64, **gqa),
        # continuous batching: most requests decode, some prefill odd chunks; narrow heads, odd pages
        dict(name="swa_mixed", op="swa", batch=24, new=777, kind="mixed", ctx=8190, window=1024, page=48,
             hq=16, hkv=2, d=64),
        # SA decoding at the benchmark's window, sigma of the full length
        dict(name="sa_decode", op="sa", batch=64, new=1, kind="decode", ctx=32768, cap=32768, window=128, page=64, **gqa),
        # SA over chunks of prompts, wide window, heads not shared
        dict(name="sa_chunk", op="sa", batch=3, new=501, kind="chunk", ctx=12000, cap=16384, window=256, page=32,
             hq=16, hkv=16, d=64),
        # one token of a batch of users through the gated layer
        dict(name="gated_decode", op="gated", batch=33, new=1, kind="decode", ctx=16384, cap=16384, window=128,
             window_swa=128, page=16, **gqa),
        # a prompt chunk through the gated layer
        dict(name="gated_chunk", op="gated", batch=2, new=1024, kind="chunk", ctx=16384, cap=32768, window=128,
             window_swa=256, page=64, **gqa),
        # the plan of a decoding step
        dict(name="plan_decode", op="plan", batch=64, new=1, kind="decode", ctx=32768, page=16),
        # the plan of a large offline batch of prompts
        dict(name="plan_prompts", op="plan", batch=1500, new=901, kind="mixed", ctx=5000, page=16),
        # one token of each user into the cache
        dict(name="append_decode", op="append", batch=128, new=1, kind="decode", ctx=4096, page=16, rope=True, **gqa),
        # prompts into the cache, queries, keys and values as slices of one projection
        dict(name="append_prompts", op="append", batch=9, new=4096, kind="chunk", ctx=65536, page=64, rope=True, **gqa),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = dict(op=rng.choice(["swa", "swa", "sa", "gated", "plan", "append"]))
        c["kind"] = rng.choice(["decode", "chunk", "mixed"])
        c["page"] = rng.choice([8, 16, 32, 48, 64, 100, 128, 256])
        c["batch"] = _log(rng, 1, 1500) if c["op"] == "plan" else _log(rng, 1, 200 if c["kind"] == "decode" else 24)
        c["new"] = 1 if c["kind"] == "decode" else _log(rng, 2, 2048)
        c["ctx"] = max(c["new"], _log(rng, 60, 32768))
        if c["op"] != "plan":
            c["hkv"] = rng.choice([1, 2, 4, 8, 16])
            c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 4, 8] if c["hkv"] < 16 else [1, 2])
            c["d"] = rng.choice([64, 128])
        if c["op"] == "append":
            c["rope"] = rng.random() < 0.7
        if c["op"] == "swa":
            c["window"] = rng.choice([_log(rng, 16, 4096), 1 << 20])
        if c["op"] in ("sa", "gated"):
            c["window"] = _log(rng, 8, 1024)
            c["cap"] = c["ctx"] + rng.randrange(0, c["ctx"])
        if c["op"] == "gated":
            c["window_swa"] = _log(rng, 16, 1024)
        w = work(c)
        rows = c["batch"] * c["new"] if c["kind"] != "decode" else c["batch"]
        pairs = c["batch"] * c.get("hq", 1) * c["new"] * c["ctx"]
        keys = c["batch"] * c["ctx"] * c.get("hkv", 1) * c.get("d", 1)
        near = rows * (c.get("window", 0) + 1) * c.get("hkv", 1) * c.get("d", 1)
        if c["op"] in ("sa", "gated") and near > 1.2e9:
            continue
        if c["op"] in ("swa", "gated") and (pairs > 2.2e9 or keys > 1.2e9):
            continue
        if c["op"] == "plan" and rows > 6e5:
            continue
        if c["op"] == "append" and rows * (c["hq"] + 2 * c["hkv"]) * c["d"] > 1.2e8:
            continue
        if keys > 2e9 or w["bytes"] > 3.5e9 or w["flops"] > 1e12:
            continue
        return c


def _lengths(case):
    """(new tokens, tokens in all) of each request: the same for every seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new, total = [], []
    for b in range(case["batch"]):
        n = case["new"]
        if case["kind"] == "mixed" and b % 4:
            n = 1
        elif case["kind"] != "decode" and b:
            n = rng.randint((n + 1) // 2, n)
        longest = case["ctx"]
        new.append(n)
        total.append(longest if b == 0 else rng.randint(min(longest, max(n, longest // 8)), longest))
    return new, total


def _pages(case, total):
    return [-(-t // case["page"]) for t in total]


# ------------------------------------------------------------------ inputs

def _tables(case, total, g):
    """Block tables (unused entries -1) over a shuffled pool of pages, some of them free."""
    need = torch.tensor(_pages(case, total))
    width, used = int(need.max()) + 2, int(need.sum())
    num_pages = used + 8 + used // 16
    ids = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    need = need.cuda()
    col = torch.arange(width, device="cuda")[None, :]
    mine = col < need[:, None]
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
    table[mine] = ids[:used]
    return table, ids, num_pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, total = _lengths(case)
    b, page = case["batch"], case["page"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    s = dict(case=case, op=case["op"], page=page, max_new=max(new), max_len=max(total))
    if case["op"] == "plan":
        cached = [t - n for t, n in zip(total, new)]
        table, ids, num_pages = _tables(case, cached, g)
        width = max(_pages(case, total)) + 2
        used = sum(_pages(case, cached))
        want = sum(_pages(case, total)) - used
        free = torch.randperm(want + 100, generator=g, device="cuda").to(torch.int32) + num_pages
        s |= dict(new_lens=i32(new), cached_lens=i32(cached), num_free=i32([want + 61]), free=free,
                  table=torch.nn.functional.pad(table, (0, max(0, width - table.shape[1])), value=-1).contiguous(),
                  num_pages=num_pages + want + 100, max_tokens=sum(new) + 7)
        return s
    table, _, num_pages = _tables(case, total, g)
    t, hq, hkv, d = sum(new), case["hq"], case["hkv"], case["d"]
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    starts = [0]
    starts += torch.tensor(new).cumsum(0).tolist()
    s |= dict(table=table, q_start=i32(starts), seq_lens=i32(total), k_cache=normal(num_pages, page, hkv, d),
              v_cache=normal(num_pages, page, hkv, d))
    if case["op"] == "append":
        qkv = normal(t, hq + 2 * hkv, d)  # one projection's output, cut into its parts
        s |= dict(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
        req = torch.repeat_interleave(torch.arange(b, device="cuda"), i32(new).long())
        pos = torch.arange(t, device="cuda") - s["q_start"].long()[req] + (s["seq_lens"] - i32(new)).long()[req]
        s["slots"] = (table[req, pos // page] * page + pos % page).to(torch.int32)
        s["positions"] = pos.to(torch.int32)
        return s
    s["q"] = normal(t, hq, d) * 2  # scores of a standard deviation of two
    if case["op"] in ("sa", "gated"):
        cap = case["cap"]
        perm = torch.argsort(torch.rand(b, cap, generator=g, device="cuda"), dim=1)
        s["perm"] = perm.to(torch.int32)
        s["inv_perm"] = torch.argsort(perm, dim=1).to(torch.int32)
    if case["op"] == "gated":
        s["gate_sa"] = torch.randn(t, hq, generator=g, device="cuda")
        s["gate_swa"] = torch.randn(t, hq, generator=g, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

ROPE_BASE = 10000.0


def run(s):
    op = s["op"]
    if own:
        import stochastic_sliding_window_gb300 as sa
        c = s["case"]
        if op == "plan":
            plan = sa.paged_plan(s["new_lens"], s["cached_lens"], s["table"], s["free"], s["num_free"],
                                 page_size=s["page"], num_pages=s["num_pages"], max_tokens=s["max_tokens"])
            return dict(table=s["table"], q_start=plan.q_start, seq_lens=plan.seq_lens, slots=plan.slots,
                        positions=plan.positions, counts=plan.counts)
        if op == "append":
            q = sa.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                                rope_base=ROPE_BASE if c["rope"] else 0.0, q=s["q"] if c["rope"] else None)
            return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], **({"q": q} if c["rope"] else {}))
        where = (s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["seq_lens"])
        if op == "swa":
            return sa.swa_paged_forward(*where, window=c["window"], max_new=s["max_new"])
        if op == "sa":
            return sa.sa_paged_forward(*where, s["perm"], s["inv_perm"], window=c["window"], max_new=s["max_new"])
        return sa.sa_swa_gated_paged_forward(*where, s["perm"], s["inv_perm"], s["gate_sa"], s["gate_swa"],
                                             window=c["window"], window_swa=c["window_swa"], max_new=s["max_new"])
    if op == "plan":
        return _plain_plan(s)
    if op == "append":
        return _plain_append(s)
    if op == "swa":
        return _plain_swa(s, s["case"]["window"]).to(torch.bfloat16)
    if op == "sa":
        return _plain_sa(s).to(torch.bfloat16)
    y = torch.sigmoid(s["gate_sa"])[..., None] * _plain_sa(s)
    y = y + torch.sigmoid(s["gate_swa"])[..., None] * _plain_swa(s, s["case"]["window_swa"])
    return y.to(torch.bfloat16)


def _plain_plan(s):
    n, c, page, cap = s["new_lens"].long(), s["cached_lens"].long(), s["page"], s["max_tokens"]
    total = c + n
    owned, need = (c + page - 1) // page, (total + page - 1) // page
    take = need - owned
    q_end, p_end = n.cumsum(0), take.cumsum(0)
    q_start, p_start = q_end - n, p_end - take
    col = torch.arange(s["table"].shape[1], device=n.device)[None, :]
    fresh = (col >= owned[:, None]) & (col < need[:, None])
    from_top = (p_start[:, None] + col - owned[:, None]).clamp(0, s["free"].numel() - 1)
    at = (s["num_free"].long() - 1 - from_top).clamp(min=0)
    table = torch.where(fresh, s["free"][at], s["table"])
    t = torch.arange(cap, device=n.device)
    live = t < q_end[-1]
    req = torch.searchsorted(q_end, t, right=True).clamp(max=n.numel() - 1)
    pos = t - q_start[req] + c[req]
    pos = torch.where(live, pos, 0)
    slot = table[req, pos // page].long() * page + pos % page
    zero = torch.zeros(1, dtype=torch.long, device=n.device)
    taken = p_end[-1:]
    s["table"].copy_(table)
    i32 = lambda x: x.to(torch.int32)
    return dict(table=s["table"], q_start=i32(torch.cat([zero, q_end])), seq_lens=i32(total),
                slots=i32(torch.where(live, slot, -1)), positions=i32(torch.where(live, pos, -1)),
                counts=i32(torch.cat([q_end[-1:], taken, s["num_free"].long() - taken])))


def _rotate(x, positions):
    """Pairs (x_k, x_{k + d/2}) turned by position * base^(-2k/d); the angles in 64 bits, the rest in 32."""
    half = x.shape[-1] // 2
    theta = ROPE_BASE ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    a = positions.double()[:, None] * theta[None, :]
    a = (a - 2 * math.pi * torch.round(a / (2 * math.pi))).float()[:, None, :]
    lo, hi = x[..., :half].float(), x[..., half:].float()
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1).to(x.dtype)


def _plain_append(s):
    rope = s["case"]["rope"]
    hkv, d = s["k"].shape[1:]
    at = s["slots"].long()
    s["k_cache"].view(-1, hkv, d)[at] = _rotate(s["k"], s["positions"]) if rope else s["k"]
    s["v_cache"].view(-1, hkv, d)[at] = s["v"]
    out = dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    if rope:
        out["q"] = _rotate(s["q"], s["positions"])
    return out


def _where(s):
    """Request and position of each new token."""
    t = torch.arange(s["q"].shape[0], device=s["q"].device)
    req = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    return req, t - s["q_start"].long()[req + 1] + s["seq_lens"].long()[req]


def _plain_swa(s, window):
    q, (hkv, d) = s["q"].float(), s["k_cache"].shape[2:]
    hq, b = q.shape[1], s["seq_lens"].numel()
    first = (s["seq_lens"] - s["q_start"].diff()).long()  # the first new token's position
    keep = min(s["max_len"], window + s["max_new"])  # no row reaches further back than this
    base = (s["seq_lens"].long() - keep).clamp(min=0)
    key = base[:, None] + torch.arange(keep, device=q.device)[None, :]  # [b, keys]
    live = key < s["seq_lens"][:, None]
    key = torch.where(live, key, 0)
    slot = torch.gather(s["table"].long(), 1, key // s["page"]) * s["page"] + key % s["page"]
    k = s["k_cache"].view(-1, hkv, d)[slot].float()  # [b, keys, hkv, d]
    v = s["v_cache"].view(-1, hkv, d)[slot].float()
    req, pos = _where(s)
    i = pos - first[req]
    wide = torch.zeros(b, s["max_new"], hq, d, device=q.device)
    wide[req, i] = q / math.sqrt(d)
    wide = wide.view(b, s["max_new"], hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    score = (wide @ k.permute(0, 2, 3, 1)).view(b, hkv, hq // hkv, s["max_new"], keep)
    at = first[:, None, None] + torch.arange(s["max_new"], device=q.device)[None, :, None]
    ok = live[:, None, :] & (key[:, None, :] <= at) & (key[:, None, :] > at - window)
    score = score.masked_fill_(~ok[:, None, None], -1e30)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    y = p.view(b, hkv, -1, keep) @ v.permute(0, 2, 1, 3)
    y = y.view(b, hkv, hq // hkv, s["max_new"], d) / total
    return y.permute(0, 3, 1, 2, 4).reshape(b, s["max_new"], hq, d)[req, i]


def _plain_sa(s):
    q, (hkv, d) = s["q"].float(), s["k_cache"].shape[2:]
    t, hq = q.shape[:2]
    h, cap = s["case"]["window"] // 2, s["perm"].shape[1]
    req, pos = _where(s)
    p = s["inv_perm"].long()[req, pos][:, None] + torch.arange(-h, h + 1, device=q.device)[None, :]
    token = s["perm"].long()[req[:, None], p.clamp(0, cap - 1)]
    ok = (p >= 0) & (p < cap) & (token <= pos[:, None])
    token = torch.where(ok, token, 0)
    slot = s["table"].long()[req[:, None], token // s["page"]] * s["page"] + token % s["page"]
    k = s["k_cache"].view(-1, hkv, d)[slot].float().transpose(1, 2)  # [t, hkv, keys, d]
    v = s["v_cache"].view(-1, hkv, d)[slot].float().transpose(1, 2)
    score = (q.view(t, hkv, hq // hkv, d) / math.sqrt(d)) @ k.transpose(2, 3)
    score = score.masked_fill(~ok[:, None, None, :], -1e30)
    w = (score - score.amax(-1, keepdim=True)).exp()
    return ((w @ v) / w.sum(-1, keepdim=True)).reshape(t, hq, d)


# ------------------------------------------------------------------ floors

def work(case):
    new, total = _lengths(case)
    t = sum(new)
    if case["op"] == "plan":
        cached = [a - n for a, n in zip(total, new)]
        grown = sum(_pages(case, total)) - sum(_pages(case, cached))
        return dict(bytes=16 * case["batch"] + 8 * t + 8 * grown + 4 * case["batch"], flops=0)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        heads = 2 * hkv + (hq if case["rope"] else 0)
        return dict(bytes=t * (heads * d * 4 + 8), flops=t * (hq + hkv) * d * 3 if case["rope"] else 0)
    small = t * hq * d * 4 + 12 * case["batch"]  # q and out, lengths
    keys = pairs = 0.0
    for n, length in zip(new, total):
        c = length - n
        far = near = 0.0
        if case["op"] in ("swa", "gated"):
            w = case["window"] if case["op"] == "swa" else case["window_swa"]
            far = length - max(0, c - w + 1)  # keys that some new token attends
            grow = max(0, min(n, w - 1 - c))  # new tokens whose window reaches the start
            pairs += grow * c + grow * (grow + 1) / 2 + (n - grow) * min(w, length)
        if case["op"] in ("sa", "gated"):
            side = 2 * (case["window"] // 2)
            each = 1 + min(side, case["cap"] - 1) * (c + (n - 1) / 2) / max(1, case["cap"] - 1)
            near = min(length, n * each)
            pairs += n * each
        keys += max(far, near)
    table = 4 * sum(_pages(case, total)) if case["op"] == "swa" else 0
    gates = 8 * t * hq if case["op"] == "gated" else 0
    return dict(bytes=keys * hkv * d * 4 + small + gates + min(table, 4 * keys / case["page"] + 4 * len(new)),
                flops=pairs * hq * d * 4)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    new, total = _lengths(case)
    page = case["page"]
    if case["op"] == "plan":
        table, free = s["table"].tolist(), s["free"].tolist()
        top = int(s["num_free"]) - 1
        taken, slots, positions, starts = 0, [], [], [0]
        for b, (n, length) in enumerate(zip(new, total)):
            for p in range(length - n, length):
                if p % page == 0:  # the first row of a page that nobody held
                    table[b][p // page] = free[top - taken]
                    taken += 1
                slots.append(table[b][p // page] * page + p % page)
                positions.append(p)
            starts.append(starts[-1] + n)
        pad = [-1] * (s["max_tokens"] - len(slots))
        i32 = lambda x: torch.tensor(x, dtype=torch.int32)
        return dict(table=i32(table), q_start=i32(starts), seq_lens=i32(total), slots=i32(slots + pad),
                    positions=i32(positions + pad), counts=i32([starts[-1], taken, top + 1 - taken]))
    if case["op"] == "append":
        turn = lambda x: x.double()
        if case["rope"]:
            half = case["d"] // 2
            freq = torch.exp(-math.log(ROPE_BASE) * torch.arange(half, dtype=torch.float64, device="cuda") / half)
            z = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), s["positions"].double()[:, None, None] * freq)

            def turn(x):
                y = torch.complex(x[..., :half].double(), x[..., half:].double()) * z
                return torch.cat([y.real, y.imag], -1)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for cache, rows in ((kc, turn(s["k"])), (vc, s["v"].double())):
            cache[(s["slots"] // page).long(), (s["slots"] % page).long()] = rows
        return dict(k_cache=kc, v_cache=vc, **({"q": turn(s["q"])} if case["rope"] else {}))
    if work(case)["flops"] > 4e12:
        return None
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.empty(sum(new), hq, d, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(new, total)):
        rows = s["table"][b, : -(-length // page)].long()
        k = s["k_cache"][rows].reshape(-1, hkv, d)[:length].double()
        v = s["v_cache"][rows].reshape(-1, hkv, d)[:length].double()
        for lo in range(0, n, 256):  # some rows at a time
            i = torch.arange(lo, min(n, lo + 256), device="cuda")
            pos = (length - n + i)[:, None]
            j = torch.arange(length, device="cuda")[None, :]
            q = s["q"][at + i].double().view(len(i), hkv, hq // hkv, d)
            first = 0
            if case["op"] == "swa":  # keys before every row's window are left out
                first = max(0, length - n + lo - case["window"] + 1)
            score = torch.einsum("ihgd,jhd->higj", q, k[first:]) / math.sqrt(d)

            def attend(seen):
                p = torch.softmax(torch.where(seen[None, :, None, first:], score, -math.inf), -1)
                return torch.einsum("higj,jhd->ihgd", p, v[first:]).reshape(len(i), hq, d)
            y = 0.0
            causal = j <= pos
            if case["op"] in ("sa", "gated"):
                place = s["inv_perm"][b, :length].long()
                y_sa = attend(causal & ((place[None, :] - place[pos]).abs() <= case["window"] // 2))
                y = y_sa if case["op"] == "sa" else y_sa / (1 + torch.exp(-s["gate_sa"][at + i].double()))[..., None]
            if case["op"] in ("swa", "gated"):
                w = case["window"] if case["op"] == "swa" else case["window_swa"]
                y_swa = attend(causal & (j > pos - w))
                y = y_swa if case["op"] == "swa" else y + y_swa / (1 + torch.exp(-s["gate_swa"][at + i].double()))[..., None]
            out[at + i] = y
        at += n
    return out
