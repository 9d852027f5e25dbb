"""Cases of the bounded-cache serving operators: attention over a shared prefix, attention mass, cache eviction.

A batch of sequences decodes behind one long prefix (a system prompt) that is stored once; every sequence's own cache
rows follow it.  Three operators keep such a batch within a fixed memory:

  attn_shared  one layer's attention of all sequences: keys [shared rows | own cache rows | new rows];
  attn_mass    the attention weight that the step's accepted tokens gave to every own cache row, added to a running sum;
  kv_evict     own caches longer than a budget give up the rows with the least mass, in place.

`run` computes them in plain torch, or through the library where `own` is set.  Sizes follow the library's own
configurations (Qwen2.5-1.5B, Qwen3-8B and Qwen3-32B shapes, draft lengths 1 to 16).
"""
import math
import random

import torch

own = False

DEV = "cuda"
PAGE = 64
HYBRID, CAUSAL = 0, 1


# ---- cases -------------------------------------------------------------------------------------------------------

def _attn(name, B, Hq, Hkv, D, k, R, S, lo, hi, paged=False):
    """k > 0: the hybrid decode mask of draft length k (R = k (k + 2) rows); k = 0: R causal rows."""
    return dict(name=name, op="attn_shared", B=B, Hq=Hq, Hkv=Hkv, D=D, k=k, R=k * (k + 2) if k else R, S=S, lo=lo,
                hi=hi, paged=paged, lens=7)


def _mass(name, L, B, Hq, Hkv, D, R, lo, hi, decay=1.0, full=False, paged=False):
    """R: rows the queries hold; the last row_count[b] <= R rows of a cache asked (all R where `full`)."""
    return dict(name=name, op="attn_mass", L=L, B=B, Hq=Hq, Hkv=Hkv, D=D, R=R, lo=lo, hi=hi, decay=decay, full=full,
                paged=paged, lens=7)


def _evict(name, L, B, Hkv, D, lo, hi, budget, sink, recent, paged=False):
    return dict(name=name, op="kv_evict", L=L, B=B, Hkv=Hkv, D=D, lo=lo, hi=hi, budget=budget, sink=sink,
                recent=recent, paged=paged, lens=7)


def listed():
    return [
        # the smallest configuration's decode step, two sequences behind a short prompt: launch latency
        _attn("shared tiny k4", 2, 2, 1, 64, 4, 0, 128, 1, 128),
        # plain token-by-token decoding of a batch behind one system prompt
        _attn("shared 8b one token b16", 16, 32, 8, 128, 0, 1, 4096, 1, 512),
        # short drafts, six query heads per KV head, a prompt that ends inside a tile, paged
        _attn("shared 1.5b k4 b8 paged", 8, 12, 2, 128, 4, 0, 1001, 64, 1024, paged=True),
        # the headline decode step as a batch of eight
        _attn("shared 8b k8 b8", 8, 32, 8, 128, 8, 0, 4096, 16, 1024),
        # the longest drafts over a long shared document: the compute-bound end
        _attn("shared 32b k16 b2", 2, 64, 8, 128, 16, 0, 16384, 512, 2048),
        # the smallest configuration after one step
        _mass("mass tiny", 1, 2, 2, 1, 64, 4, 5, 128),
        # every layer of the headline step, up to eight accepted drafts
        _mass("mass 8b all layers", 36, 1, 32, 8, 128, 8, 4096, 4096, decay=0.98),
        # a prompt's last rows asked once, ragged and paged: many query rows per key
        _mass("mass 1.5b prompt rows paged", 4, 3, 12, 2, 128, 77, 500, 4096, full=True, paged=True),
        # long caches and long drafts
        _mass("mass 32b long", 16, 1, 64, 8, 128, 16, 16384, 16384),
        # a decode step's trim: a handful of rows over the budget in every head of every layer
        _evict("evict 8b steady", 36, 1, 8, 128, 2056, 2056, 2048, 4, 128),
        # ragged batch over paged caches, some under the budget
        _evict("evict 1.5b ragged paged", 28, 4, 2, 128, 300, 1500, 1000, 1, 77, paged=True),
        # a long prompt cut down to the budget once
        _evict("evict 32b prompt", 16, 1, 8, 128, 16384, 16384, 4096, 16, 512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attn_shared", "attn_mass", "kv_evict"])
    Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128])
    G = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8])
    lens, paged = rng.randrange(1 << 20), rng.random() < 0.4
    if op == "attn_shared":
        while True:
            k = rng.choice([0, 1, 2, 3, 4, 5, 6, 8, 11, 16])
            R = k * (k + 2) if k else _log_int(rng, 1, 100)
            B, S, hi = _log_int(rng, 1, 48), _log_int(rng, 1, 20000), _log_int(rng, 1, 3000)
            if 4.0 * B * R * Hkv * G * D * (S + hi) <= 2.0e11:
                break
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, k=k, R=R, S=S, lo=rng.randint(0, hi), hi=hi, paged=paged,
                    lens=lens)
    if op == "attn_mass":
        while True:
            L, B, R, hi = _log_int(rng, 1, 40), _log_int(rng, 1, 12), _log_int(rng, 1, 96), _log_int(rng, 100, 20000)
            if L * B * Hkv * hi * D <= 2.5e8 and 2.0 * L * B * Hkv * G * R * hi * D <= 6e10:
                break
        return dict(op=op, L=L, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, R=R, lo=rng.randint(R, max(R, hi)), hi=max(R, hi),
                    decay=rng.choice([1.0, 0.95]), full=rng.random() < 0.3, paged=paged, lens=lens)
    while True:
        L, B, hi = _log_int(rng, 1, 40), _log_int(rng, 1, 12), _log_int(rng, 100, 20000)
        if L * B * Hkv * hi * D <= 2.5e8:
            break
    budget = rng.randint(hi // 4, hi - 1)
    recent = rng.randint(0, min(600, budget // 2))
    return dict(op=op, L=L, B=B, Hkv=Hkv, D=D, lo=rng.randint(budget // 2, hi), hi=hi, budget=budget,
                sink=rng.randint(0, min(32, budget - recent)), recent=recent, paged=paged, lens=lens)


def _lengths(c):
    """Own cache lengths, the longest among them (part of the case: the same for every seed)."""
    r = random.Random(c["lens"])
    return [c["hi"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["B"] - 1)]


def _row_counts(c):
    """Rows of the step that count: accept lengths 0..R, the first of them R."""
    r = random.Random(c["lens"] + 1)
    return [c["R"] if c["full"] or b == 0 else r.randint(0, c["R"]) for b in range(c["B"])]


# ---- inputs ------------------------------------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _caches(g, n, B, Hkv, P_max, D, lens, paged, spare=0):
    """n caches: contiguous [n, B, Hkv, P_max, D] with NaN past each length, or pools [n, pages, Hkv, 64, D] with a
    permuted table [B, P_max / 64] (and `spare` more pages for the shared prefix, whose ids come second)."""
    if not paged:
        c = torch.empty((n, B, Hkv, P_max, D), device=DEV, dtype=torch.bfloat16)
        for i in range(n):
            c[i] = _normal(g, B, Hkv, P_max, D)
        for b in range(B):
            c[:, b, :, lens[b]:] = float("nan")
        return c
    per = P_max // PAGE
    c = torch.empty((n, B * per + spare, Hkv, PAGE, D), device=DEV, dtype=torch.bfloat16)
    for i in range(n):
        c[i] = _normal(g, B * per + spare, Hkv, PAGE, D)
    return c


def _pad_rows(n):
    return (n + PAGE - 1) // PAGE * PAGE


def _pointers(t):
    return torch.tensor([t[i].data_ptr() for i in range(t.shape[0])], dtype=torch.int64, device=DEV)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    lens = _lengths(c)
    P_max = _pad_rows(max(lens) + 16)
    s = dict(c=c, P_max=P_max, status=torch.zeros(1, dtype=torch.int32, device=DEV),
             prefix_len=torch.tensor(lens, dtype=torch.int32, device=DEV))
    spare = _pad_rows(c.get("S", 0)) // PAGE if c["paged"] else 0
    if c["paged"]:
        pages = torch.randperm(B * (P_max // PAGE) + spare, generator=g, device=DEV).to(torch.int32)
        s["table"] = pages[:B * (P_max // PAGE)].reshape(B, -1).contiguous()
        s["shared_table"] = pages[B * (P_max // PAGE):].contiguous()
        s["num_pages"] = pages.numel()
    if c["op"] == "attn_shared":
        Hq, R, S = c["Hq"], c["R"], c["S"]
        s["q"], s["kn"], s["vn"] = 1.5 * _normal(g, B, R, Hq, D), _normal(g, B, R, Hkv, D), _normal(g, B, R, Hkv, D)
        s["kc"] = _caches(g, 1, B, Hkv, P_max, D, lens, c["paged"], spare)[0]
        s["vc"] = _caches(g, 1, B, Hkv, P_max, D, lens, c["paged"], spare)[0]
        if not c["paged"]:
            s["ks"], s["vs"] = _normal(g, Hkv, S, D), _normal(g, Hkv, S, D)
        s["shared_len"] = torch.tensor([S], dtype=torch.int32, device=DEV)
        s["out"] = torch.empty((B, R, Hq, D), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((B, R, Hq), dtype=torch.float32, device=DEV)
    elif c["op"] == "attn_mass":
        L, Hq, R = c["L"], c["Hq"], c["R"]
        s["q"] = 1.5 * _normal(g, L, B, R, Hq, D)
        s["kc"] = _caches(g, L, B, Hkv, P_max, D, lens, c["paged"])
        s["row_count"] = torch.tensor(_row_counts(c), dtype=torch.int32, device=DEV)
        # the step's own log-sum-exps: of about the size that rows of these scores have (scores ~ N(0, 1.5^2))
        s["lse"] = (s["prefix_len"].float().log()[None, :, None, None] + 1.125
                    + 0.3 * torch.randn((L, B, R, Hq), generator=g, device=DEV)).contiguous()
        s["mass"] = torch.rand((L, B, Hkv, P_max), generator=g, device=DEV)
        s["ptr_q"], s["ptr_k"], s["ptr_lse"], s["ptr_mass"] = map(_pointers, (s["q"], s["kc"], s["lse"], s["mass"]))
    else:
        L = c["L"]
        s["kc"] = _caches(g, L, B, Hkv, P_max, D, lens, c["paged"])
        s["vc"] = _caches(g, L, B, Hkv, P_max, D, lens, c["paged"])
        for t in (s["kc"], s["vc"]):  # finite everywhere: whole caches come back
            t.nan_to_num_(nan=0.0)
        # accumulated attention weight: many small sums, few large ones, and rows that no token has looked at yet
        m = torch.randn((L, B, Hkv, P_max), generator=g, device=DEV).mul_(2.0).exp_()
        s["mass0"] = torch.where(torch.rand((L, B, Hkv, P_max), generator=g, device=DEV) < 0.02, 0.0, m)
        s["mass"] = s["mass0"].clone()
        s["len0"] = s["prefix_len"].clone()
        s["ptr_k"], s["ptr_v"], s["ptr_mass"] = map(_pointers, (s["kc"], s["vc"], s["mass"]))
    return s


# ---- plain forms -------------------------------------------------------------------------------------------------

def _rows_of(pool, table):
    """Pages [.., num_pages, Hkv, 64, D] of a table [B, n] as contiguous caches [.., B, Hkv, 64 n, D]."""
    x = pool[..., table.long(), :, :, :]  # [.., B, n, Hkv, 64, D]
    return x.transpose(-4, -3).flatten(-3, -2)


def _visible(k, R):
    """[R, R] bool: which new keys a new row sees."""
    r = torch.arange(R, device=DEV)
    row, key = r[:, None], r[None, :]
    if k == 0:
        return key <= row
    group_r, group_n = (row - k) // k, (key - k) // k
    draft_row, draft_key = row < k, key < k
    return torch.where(draft_row, key <= row, torch.where(draft_key, key < group_r, group_n == group_r))


def _plain_attn(s):
    c = s["c"]
    B, Hq, Hkv, D, R, S, P = c["B"], c["Hq"], c["Hkv"], c["D"], c["R"], c["S"], s["P_max"]
    G = Hq // Hkv
    if c["paged"]:
        kc, vc = _rows_of(s["kc"], s["table"]), _rows_of(s["vc"], s["table"])
        ks, vs = (_rows_of(t, s["shared_table"][None])[0, :, :S] for t in (s["kc"], s["vc"]))
    else:
        kc, vc, ks, vs = s["kc"], s["vc"], s["ks"], s["vs"]
    scale = 1.0 / math.sqrt(D)
    q = s["q"].float().reshape(B, R, Hkv, G, D).permute(2, 0, 1, 3, 4)  # [Hkv, B, R, G, D]
    held = torch.arange(P, device=DEV)[None] < s["prefix_len"][:, None]  # [B, P]
    kc = kc.float().masked_fill(~held[:, None, :, None], 0.0).transpose(0, 1)  # [Hkv, B, P, D]
    vc = vc.float().masked_fill(~held[:, None, :, None], 0.0).transpose(0, 1)
    kn, vn = s["kn"].float().permute(2, 0, 1, 3), s["vn"].float().permute(2, 0, 1, 3)  # [Hkv, B, R, D]
    qb = q.reshape(Hkv, B, R * G, D)
    low = float("-inf")
    a = (q.reshape(Hkv, B * R * G, D) @ ks.float().mT).reshape(Hkv, B, R, G, S)
    b = (qb @ kc.mT).reshape(Hkv, B, R, G, P).masked_fill(~held[None, :, None, None], low)
    d = (qb @ kn.mT).reshape(Hkv, B, R, G, R).masked_fill(~_visible(c["k"], R)[None, None, :, None], low)
    x = torch.cat([a, b, d], -1).mul_(scale)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x[..., :S].reshape(Hkv, B * R * G, S) @ vs.float()).reshape(Hkv, B, R * G, D)
    o = o + x[..., S:S + P].reshape(Hkv, B, R * G, P) @ vc + x[..., S + P:].reshape(Hkv, B, R * G, R) @ vn
    o = o.reshape(Hkv, B, R, G, D) / total
    lse = (top + total.log()).squeeze(-1)
    return (o.permute(1, 2, 0, 3, 4).reshape(B, R, Hq, D).to(torch.bfloat16),
            lse.permute(1, 2, 0, 3).reshape(B, R, Hq))


def _plain_mass(s):
    c = s["c"]
    L, B, Hq, Hkv, D, R, P = c["L"], c["B"], c["Hq"], c["Hkv"], c["D"], c["R"], s["P_max"]
    G = Hq // Hkv
    kc = _rows_of(s["kc"], s["table"]) if c["paged"] else s["kc"]
    n, a = s["prefix_len"][:, None, None], s["row_count"][:, None, None]
    row = torch.arange(P, device=DEV)[None, None]
    r = torch.arange(R, device=DEV)[None, :, None]
    seen = (r < a) & (row < n - a + r + 1)  # [B, R, P]: the a newest tokens are the cache's last a rows
    q = s["q"].float().reshape(L, B, R, Hkv, G, D).permute(0, 1, 3, 2, 4, 5).reshape(L, B, Hkv, R * G, D)
    lse = s["lse"].reshape(L, B, R, Hkv, G).permute(0, 1, 3, 2, 4).reshape(L, B, Hkv, R * G, 1)
    w = (q @ kc.float().mT).mul_(1.0 / math.sqrt(D)).sub_(lse).exp_().reshape(L, B, Hkv, R, G, P)
    w = w.masked_fill_(~seen[None, :, None, :, None], 0.0).sum((3, 4))  # [L, B, Hkv, P]
    row, n, a = row[0][None], n[:, 0], a[:, 0]  # [1, 1, P], [B, 1]
    old = (row[0] < n - a)[None, :, None]
    new = ((row[0] >= n - a) & (row[0] < n))[None, :, None]
    m = s["mass"]
    m.copy_(torch.where(old, c["decay"] * m + w, torch.where(new, w, m)))
    return m


def _plain_evict(s):
    c = s["c"]
    L, B, Hkv, D, P = c["L"], c["B"], c["Hkv"], c["D"], s["P_max"]
    budget, sink, recent = c["budget"], c["sink"], c["recent"]
    s["mass"].copy_(s["mass0"])
    n = s["len0"].long()[None, :, None, None]  # [1, B, 1, 1]
    m = s["mass"]
    row = torch.arange(P, device=DEV)[None, None, None]
    zone = budget - recent  # rows [sink, zone) hold the heaviest, [zone, budget) the newest
    cand = (row >= sink) & (row < n - recent)
    order = torch.where(cand, m, -1.0).argsort(dim=-1, descending=True, stable=True)  # heaviest first, ties by index
    rank = torch.empty_like(order).scatter_(-1, order, row.expand_as(order))
    keep = cand & (rank < zone - sink)
    hole = (cand & ~keep & (row < zone)).long()
    tail = keep & (row >= zone)  # survivors that have to move
    by_index = (~tail).long().argsort(dim=-1, stable=True)  # the survivors first, ascending
    src = row + torch.zeros_like(order)
    src = torch.where(hole.bool(), by_index.gather(-1, (hole.cumsum(-1) - 1).clamp_min(0)), src)
    src = torch.where((row >= zone) & (row < budget), row + n - budget, src)
    src = torch.where(n > budget, src, row)
    moved = m.gather(-1, src)
    m.copy_(moved)
    at = src[..., None].expand(L, B, Hkv, P, D)
    if c["paged"]:
        k, v = (_rows_of(t, s["table"]).gather(3, at) for t in (s["kc"], s["vc"]))
        t = s["table"].long()
        s["kc"][:, t] = k.reshape(L, B, Hkv, -1, PAGE, D).transpose(2, 3)
        s["vc"][:, t] = v.reshape(L, B, Hkv, -1, PAGE, D).transpose(2, 3)
    else:
        s["kc"].copy_(s["kc"].gather(3, at))
        s["vc"].copy_(s["vc"].gather(3, at))
    s["prefix_len"].copy_(s["len0"].clamp_max(budget))
    return s["kc"], s["vc"], m, s["prefix_len"]


# ---- the library's calls -----------------------------------------------------------------------------------------

def _own_attn(s):
    from ar_lm_decoding_b200 import abi
    c = s["c"]
    B, Hq, Hkv, D, R, k, S, P = c["B"], c["Hq"], c["Hkv"], c["D"], c["R"], c["k"], c["S"], s["P_max"]
    if "ws" not in s:
        size = abi.tidar_attn_shared_workspace_size(B, Hq, Hkv, D, R, _pad_rows(S) if c["paged"] else S, P)
        s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    mode, scale = HYBRID if k else CAUSAL, 1.0 / math.sqrt(D)
    if c["paged"]:
        abi.tidar_attn_step_shared_paged(
            s["q"], s["kn"], s["vn"], s["kc"], s["vc"], s["shared_table"], s["shared_table"].numel(), s["shared_len"],
            s["table"], s["table"].shape[1], s["num_pages"], s["prefix_len"], B, Hq, Hkv, D, k, R, scale, mode,
            s["out"], s["lse"], s["ws"], s["ws"].numel(), s["status"])
    else:
        abi.tidar_attn_step_shared(
            s["q"], s["kn"], s["vn"], s["ks"], s["vs"], s["shared_len"], S, s["kc"], s["vc"], s["prefix_len"], B, Hq,
            Hkv, D, k, R, P, scale, mode, s["out"], s["lse"], s["ws"], s["ws"].numel(), s["status"])
    return s["out"], s["lse"]


def _paging(s):
    return (s["table"], s["table"].shape[1], s["num_pages"]) if s["c"]["paged"] else (None, 0, 0)


def _own_mass(s):
    from ar_lm_decoding_b200 import abi
    c = s["c"]
    abi.tidar_attn_mass(s["ptr_q"], s["ptr_lse"], s["ptr_k"], s["ptr_mass"], *_paging(s), s["prefix_len"],
                        s["row_count"], c["L"], c["B"], c["Hq"], c["Hkv"], c["D"], c["R"], s["P_max"],
                        1.0 / math.sqrt(c["D"]), c["decay"], s["status"])
    return s["mass"]


def _own_evict(s):
    from ar_lm_decoding_b200 import abi
    c = s["c"]
    s["mass"].copy_(s["mass0"])  # the masses and lengths of the next step: the same work in every pass
    s["prefix_len"].copy_(s["len0"])
    abi.tidar_kv_evict(s["ptr_k"], s["ptr_v"], s["ptr_mass"], *_paging(s), s["prefix_len"], c["L"], c["B"], c["Hkv"],
                       c["D"], s["P_max"], c["budget"], c["sink"], c["recent"], s["status"])
    return s["kc"], s["vc"], s["mass"], s["prefix_len"]


def run(state):
    op = state["c"]["op"]
    if own:
        return {"attn_shared": _own_attn, "attn_mass": _own_mass, "kv_evict": _own_evict}[op](state)
    return {"attn_shared": _plain_attn, "attn_mass": _plain_mass, "kv_evict": _plain_evict}[op](state)


# ---- what a pass cannot do without -------------------------------------------------------------------------------

def work(case):
    c = case
    lens, Hkv, D, B = _lengths(c), c["Hkv"], c["D"], c["B"]
    if c["op"] == "attn_shared":
        Hq, R, S, k = c["Hq"], c["R"], c["S"], c["k"]
        new = sum((r + 1) if (k == 0 or r < k) else (r - k) // k + k for r in range(R))  # visible new keys, all rows
        keys = S + sum(lens) + B * R
        return dict(bytes=4.0 * keys * Hkv * D + 4.0 * B * R * Hq * D + 4.0 * B * R * Hq,
                    flops=4.0 * D * Hq * (R * (B * S + sum(lens)) + B * new))
    if c["op"] == "attn_mass":
        L, Hq, rows = c["L"], c["Hq"], _row_counts(c)
        read = sum(n for n, a in zip(lens, rows) if a)
        return dict(bytes=L * (2.0 * read * Hkv * D + 8.0 * sum(lens) * Hkv + sum(rows) * Hq * (2.0 * D + 4)),
                    flops=L * 2.0 * D * Hq * sum(a * (n - a) + a * (a + 1) / 2 for n, a in zip(lens, rows)))
    heads, zone, total = c["L"] * Hkv, c["budget"] - c["recent"], 0.0
    for n in lens:
        if n > c["budget"]:
            cand = n - c["recent"] - c["sink"]
            moves = c["recent"] + (n - c["budget"]) * (zone - c["sink"]) / cand  # the newest rows, the filled holes
            total += heads * (4.0 * cand + moves * 2 * (2 * 2.0 * D + 4))
    # a pass also brings in the step's masses
    return dict(bytes=total + 8.0 * heads * B * _pad_rows(max(lens) + 16), flops=heads * float(sum(lens)))


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------

def _logical(s, t, layer, b):
    """Own cache of one sequence of one layer in 64 bits: [Hkv, len, D]."""
    n = int(s["prefix_len"][b]) if "len0" not in s else int(s["len0"][b])
    if not s["c"]["paged"]:
        return t[layer, b, :, :n].double()
    pages = [int(p) for p in s["table"][b, :(n + PAGE - 1) // PAGE]]
    return torch.cat([t[layer, p] for p in pages], 1)[:, :n].double()


def _exact_attn(s):
    c = s["c"]
    B, Hq, Hkv, D, R, S, k = c["B"], c["Hq"], c["Hkv"], c["D"], c["R"], c["S"], c["k"]
    G = Hq // Hkv
    out = torch.empty((B, R, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((B, R, Hq), dtype=torch.float64, device=DEV)
    if c["paged"]:
        ks, vs = (torch.cat([t[int(p)] for p in s["shared_table"]], 1)[:, :S].double() for t in (s["kc"], s["vc"]))
    else:
        ks, vs = s["ks"].double(), s["vs"].double()
    sees = torch.zeros((R, R), dtype=torch.bool)
    for r in range(R):
        if k == 0 or r < k:
            sees[r, :r + 1] = True
        else:
            j = (r - k) // k
            sees[r, :j] = True
            sees[r, k + j * k:k + j * k + k] = True
    sees = sees.to(DEV)
    for b in range(B):
        kb, vb = _logical(s, s["kc"][None], 0, b), _logical(s, s["vc"][None], 0, b)
        for h in range(Hkv):
            keys = torch.cat([ks[h], kb[h], s["kn"][b, :, h].double()])
            vals = torch.cat([vs[h], vb[h], s["vn"][b, :, h].double()])
            may = torch.cat([torch.ones((R, S + kb.shape[1]), dtype=torch.bool, device=DEV), sees], 1)
            x = torch.einsum("rgd,nd->grn", s["q"][b, :, h * G:(h + 1) * G].double(), keys) / math.sqrt(D)
            x = torch.where(may[None], x, torch.full_like(x, -math.inf))
            z = torch.logsumexp(x, -1)  # [G, R]
            lse[b, :, h * G:(h + 1) * G] = z.T
            out[b, :, h * G:(h + 1) * G] = torch.einsum("grn,nd->rgd", torch.exp(x - z[..., None]), vals)
    return out, lse


def _exact_mass(s):
    c = s["c"]
    L, B, Hkv, D, decay = c["L"], c["B"], c["Hkv"], c["D"], c["decay"]
    G = c["Hq"] // Hkv
    mass = s["mass"].double()
    rows = _row_counts(c)
    for b in range(B):
        n, a = int(s["prefix_len"][b]), rows[b]
        for layer in range(L):
            keys = _logical(s, s["kc"], layer, b)
            q = s["q"][layer, b, :a].double().reshape(a, Hkv, G, D)
            x = torch.einsum("ahgd,hnd->hgan", q, keys) / math.sqrt(D)
            x = x - s["lse"][layer, b, :a].double().reshape(a, Hkv, G).permute(1, 2, 0)[..., None]
            w = torch.exp(x)
            w[..., n - a:] = torch.tril(w[..., n - a:])  # a token sees itself and what came before it
            w = w.sum((1, 2))
            mass[layer, b, :, :n - a] = decay * mass[layer, b, :, :n - a] + w[:, :n - a]
            mass[layer, b, :, n - a:n] = w[:, n - a:]
    return mass


def _exact_evict(s):
    import numpy as np
    c = s["c"]
    budget, sink, recent = c["budget"], c["sink"], c["recent"]
    zone = budget - recent
    k, v, m = s["kc"].double(), s["vc"].double(), s["mass0"].double()
    lens = [int(x) for x in s["len0"]]
    told = s["mass0"].cpu().numpy()
    for b, n in enumerate(lens):
        if n <= budget:
            continue
        for layer in range(c["L"]):
            for h in range(c["Hkv"]):
                x = told[layer, b, h]
                at = np.arange(sink, n - recent)
                worst = at[np.lexsort((-at, x[at]))][:n - budget]  # least mass first, of equals the later row
                gone = set(worst.tolist())
                to = sorted(i for i in gone if i < zone) + list(range(zone, budget))
                of = [i for i in range(zone, n - recent) if i not in gone] + list(range(n - recent, n))
                to, of = torch.tensor(to, device=DEV), torch.tensor(of, device=DEV)
                m[layer, b, h, to] = m[layer, b, h, of]
                for t in (k, v):
                    if c["paged"]:
                        pages = s["table"][b].long()
                        t[layer, pages[to // PAGE], h, to % PAGE] = t[layer, pages[of // PAGE], h, of % PAGE]
                    else:
                        t[layer, b, h, to] = t[layer, b, h, of]
    return k, v, m, None


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn_shared": _exact_attn, "attn_mass": _exact_mass, "kv_evict": _exact_evict}[case["op"]](s)
