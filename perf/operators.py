"""Cases for measuring the operators of the paged latent cache.

Five entry points, each as a case kind below:

  split    split_mla_decode_paged: dense attention of the new tokens of each
           sequence over its paged latent cache, split over the cache's length
  window   window_mla: a prefill whose rows see a sliding window and the first
           few tokens of the sequence (sinks)
  wdecode  window_mla_decode_paged: the same mask for the new tokens of a decode
  mass     attention_mass_paged: the attention weight each cached token received
           from the new tokens, added to its running total
  evict    cache_evict_paged: keep the sinks, the most recent tokens and, of the
           rest, those of the largest running totals; compact the cache in place

``own`` selects what run() computes: False the plain form (elementary torch
operations in 32 bits, rounded once at the end), True the library's calls.
"""
import math

import torch

own = False

D, DV, BLK = 576, 512, 64       # key width, value width, tokens per cache block
SM_SCALE = 1.0 / math.sqrt(D)


def listed():
    return [
        # a single user's chat turn: the call's latency is what counts
        dict(name="split_one_short", op="split", B=1, lo=517, hi=517, nq=1, H=128),
        # a single user with the longest context the configurations name
        dict(name="split_one_long", op="split", B=1, lo=131072, hi=131072, nq=1, H=128),
        # the serving batch of the decode configuration: 64 sequences of 32768 tokens
        dict(name="split_B64_32K", op="split", B=64, lo=32768, hi=32768, nq=1, H=128),
        # a mixed batch with two tokens drafted ahead, lengths from one token on
        dict(name="split_ragged_nq2", op="split", B=33, lo=1, hi=32768, nq=2, H=128),
        # a small model's continuation of a chunked prompt, odd everywhere
        dict(name="window_small_chunk", op="window", T=203, q_pos0=5001, H=8, sinks=4, window=255),
        # a whole prompt of a large model under a window of 1024
        dict(name="window_prompt", op="window", T=8191, q_pos0=0, H=128, sinks=4, window=1024),
        # the serving batch under a window: every call touches only 2052 tokens a sequence
        dict(name="wdecode_B64", op="wdecode", B=64, lo=32768, hi=32768, nq=2, H=128, sinks=4,
             window=2048),
        # the running totals of the serving batch, after each decode step
        dict(name="mass_B64_32K", op="mass", B=64, lo=32768, hi=32768, nq=1, H=128),
        # the same for a few users of a small model with drafted tokens
        dict(name="mass_ragged_small", op="mass", B=5, lo=33, hi=9001, nq=3, H=8),
        # the serving batch brought down to half its length
        dict(name="evict_B64_half", op="evict", B=64, lo=32768, hi=32768, budget=16384, sinks=4,
             recent=2048),
        # one user's longest context brought down to a quarter
        dict(name="evict_one_long", op="evict", B=1, lo=131072, hi=131072, budget=32768, sinks=4,
             recent=1024),
        # a mixed batch where many sequences are still within the budget
        dict(name="evict_ragged", op="evict", B=19, lo=65, hi=5000, budget=1001, sinks=3,
             recent=257),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["split", "window", "wdecode", "mass", "evict"])
    H = rng.choice([8, 128, _log(rng, 1, 128)])
    if op == "window":
        T = _log(rng, 1, 8191)
        return dict(op=op, T=T, q_pos0=rng.choice([0, _log(rng, 1, 65536)]), H=H,
                    sinks=rng.choice([0, 4, rng.randint(1, 128)]), window=_log(rng, 1, 1024))
    hi = _log(rng, 2, 131072)
    B = min(_log(rng, 1, 64), max(1, 64 * 32768 // hi))
    lo = rng.choice([hi, max(1, hi // 32)])
    if op == "evict":
        budget = max(1, _log(rng, max(1, hi // 8), hi))
        sinks = rng.randint(0, min(8, budget))
        return dict(op=op, B=B, lo=lo, hi=hi, budget=budget, sinks=sinks,
                    recent=rng.randint(0, budget - sinks))
    nq = rng.choice([1, 1, 2, 3, 4])
    while nq > 1 and nq * B * hi * H > 64 * 32768 * 128:
        nq -= 1
    case = dict(op=op, B=B, lo=lo, hi=hi, nq=nq, H=H)
    if op == "wdecode":
        case.update(sinks=rng.choice([0, 4, rng.randint(1, 128)]), window=_log(rng, 1, 2048))
    return case


def _lengths(case):
    """B lengths spread evenly over the logarithm of [lo, hi]."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [min(hi, int(round(lo * (hi / lo) ** ((i + 0.5) / B)))) for i in range(B)]


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    out = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 28):          # 32-bit draws a GB at a time
        n = min(1 << 28, flat.numel() - a)
        flat[a:a + n] = torch.randn(n, generator=g, device="cuda")
    return out


def _paged(case, g):
    """Lengths in a random order, blocks at random places of the pool, and a cache
    whose first four tokens draw attention, as the first tokens of trained models do."""
    lens = torch.tensor(_lengths(case), dtype=torch.int64)
    lens = lens[torch.randperm(len(lens), generator=g, device="cuda").cpu()]
    nb = (lens + BLK - 1) // BLK
    nblk, max_blocks = int(nb.sum()), int(nb.max())
    perm = torch.randperm(nblk, generator=g, device="cuda").to(torch.int32)
    used = torch.arange(max_blocks).unsqueeze(0) < nb.unsqueeze(1)
    table = torch.full((len(lens), max_blocks), -1, dtype=torch.int32)
    table[used] = perm.cpu()
    table = table.cuda()
    kv = _randn(g, nblk, BLK, D)
    u = torch.randn(D, generator=g, device="cuda")
    u /= u.norm()
    first = table[:, 0].long()
    kv[first, :4] = (kv[first, :4].float() + 16.0 * u).bfloat16()
    return dict(kv_pool=kv, block_table=table, seq_len=lens.to(torch.int32).cuda(), u=u)


def _queries(g, u, *shape):
    q = _randn(g, *shape, D)
    flat = q.view(-1, D)
    for a in range(0, flat.shape[0], 1 << 18):
        flat[a:a + (1 << 18)] = (flat[a:a + (1 << 18)].float() + 6.0 * u).bfloat16()
    return q


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    st = dict(case)
    if op == "window":
        S = case["q_pos0"] + case["T"]
        u = torch.randn(D, generator=g, device="cuda")
        u /= u.norm()
        kv = _randn(g, S, D)
        kv[:4] = (kv[:4].float() + 16.0 * u).bfloat16()
        st.update(kv=kv, q=_queries(g, u, case["T"], case["H"]))
        return st
    st.update(_paged(case, g))
    B = case["B"]
    if op == "evict":
        ld = st["block_table"].shape[1] * BLK
        nblk = st["kv_pool"].shape[0]
        # running totals: heavy-tailed, and in steps, so that there are ties
        m = torch.exp(1.5 * torch.randn(B, ld, generator=g, device="cuda"))
        st["mass"] = torch.round(m * 256) / 256
        st["k8_pool"] = torch.randint(0, 127, (nblk, BLK, 128), generator=g, device="cuda",
                                      dtype=torch.uint8)
        st["k_scale_pool"] = torch.rand(nblk, BLK, generator=g, device="cuda") + 0.5
        st["mass_out"] = torch.zeros(B, ld, device="cuda")
        st["seq_len_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return st
    st["q"] = _queries(g, st["u"], B, case["nq"], case["H"])
    if op == "mass":
        ld = st["block_table"].shape[1] * BLK
        st["lse"] = _paged_logits(st)[1]                # what the decode call returned
        st["mass"] = torch.rand(B, ld, generator=g, device="cuda")
    return st


# -------------------------------------------------------------- plain forms

def _visible(pos, qpos, sinks, window):
    """Whether the query at qpos sees the key at pos (window 0: every earlier key)."""
    see = (pos >= 0) & (pos <= qpos)
    if window:
        see = see & ((pos < sinks) | (pos > qpos - window))
    return see


def _paged_rows(st, pos):
    """Rows of the cache at the positions pos [B, n], in 32 bits."""
    safe = pos.clamp(0, st["block_table"].shape[1] * BLK - 1)
    blk = torch.gather(st["block_table"].long(), 1, safe // BLK).clamp(min=0)
    return st["kv_pool"].view(-1, D)[blk * BLK + safe % BLK].float()


def _paged_logits(st, pos=None, sinks=0, window=0):
    """Scaled logits [B, nq, H, n] (unseen keys -inf), their lse, and the rows."""
    B, nq, H = st["q"].shape[:3]
    lens = st["seq_len"].long().view(B, 1, 1)
    if pos is None:
        pos = torch.arange(st["block_table"].shape[1] * BLK, device="cuda").expand(B, -1)
    rows = _paged_rows(st, pos)
    z = torch.bmm(st["q"].float().view(B, nq * H, D), rows.transpose(1, 2)) * SM_SCALE
    qpos = lens - nq + torch.arange(nq, device="cuda").view(1, nq, 1)
    see = _visible(pos.unsqueeze(1), qpos, sinks, window).unsqueeze(2)
    z = z.view(B, nq, H, -1).masked_fill_(~see, -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)
    lse = (m + torch.exp(z - m).sum(-1, keepdim=True).log()).squeeze(-1)
    return z, lse, rows


def _weighted(z, lse, rows):
    p = torch.exp(z - lse.unsqueeze(-1).clamp(min=-1e30))
    B, nq, H = lse.shape
    o = torch.bmm(p.view(B, nq * H, -1), rows[:, :, :DV])
    return o.view(B, nq, H, DV).bfloat16()


def _plain_split(st):
    z, lse, rows = _paged_logits(st)
    return _weighted(z, lse, rows), lse


def _plain_wdecode(st):
    nq, s, w = st["nq"], st["sinks"], st["window"]
    B = st["q"].shape[0]
    lens = st["seq_len"].long().view(B, 1)
    near = lens - nq - w + 1 + torch.arange(w + nq - 1, device="cuda").view(1, -1)
    first = torch.arange(s, device="cuda").expand(B, s)
    first = first.masked_fill(first >= near[:, :1], -1)     # counted in the window part
    z, lse, rows = _paged_logits(st, torch.cat([first, near], 1), s, w)
    return _weighted(z, lse, rows), lse


def _plain_window(st):
    q, kv, s, w, p0 = st["q"], st["kv"], st["sinks"], st["window"], st["q_pos0"]
    T, H = q.shape[:2]
    c = min(T, max(64, w))                                   # query rows of one band
    nb = (T + c - 1) // c
    qb = torch.cat([q, q.new_zeros(nb * c - T, H, D)]).float().view(nb, c * H, D)
    start = p0 + c * torch.arange(nb, device="cuda").view(nb, 1)
    near = start - w + 1 + torch.arange(c + w - 1, device="cuda").view(1, -1)
    first = torch.arange(s, device="cuda").expand(nb, s)
    first = first.masked_fill(first >= near[:, :1], -1)
    pos = torch.cat([first, near], 1)
    rows = kv[pos.clamp(0, kv.shape[0] - 1)].float()
    z = torch.bmm(qb, rows.transpose(1, 2)).mul_(SM_SCALE)
    qpos = start.view(nb, 1, 1) + torch.arange(c, device="cuda").view(1, c, 1)
    see = _visible(pos.unsqueeze(1), qpos, s, w).unsqueeze(2)
    z = z.view(nb, c, H, -1).masked_fill_(~see, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(nb, c * H, -1), rows[:, :, :DV]).view(nb, c, H, DV) / l
    lse = (m + l.log()).view(nb * c, H)[:T]
    return o.view(nb * c, H, DV)[:T].bfloat16(), lse.contiguous()


def _plain_mass(st):
    z = _paged_logits(st)[0]
    got = torch.exp(z - st["lse"].unsqueeze(-1).clamp(min=-1e30)).sum((1, 2))
    pos = torch.arange(got.shape[1], device="cuda").view(1, -1)
    n = st["seq_len"].long().view(-1, 1)
    old = torch.where(pos < n - st["nq"], st["mass"], torch.zeros_like(st["mass"]))
    st["mass"].copy_(torch.where(pos < n, old + got, st["mass"]))
    return st["mass"]


def _plain_evict(st):
    n = st["seq_len"].long().view(-1, 1)
    B, ld = st["mass"].shape
    keep = st["budget"]
    pos = torch.arange(ld, device="cuda").view(1, -1)
    fixed = (pos < st["sinks"]) | (pos >= n - st["recent"])
    rank = torch.where(fixed, math.inf, st["mass"])
    rank = torch.where(pos < n, rank, -math.inf)
    order = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :keep]
    order = torch.nn.functional.pad(order, (0, keep - order.shape[1]), value=ld)
    slot = torch.arange(keep, device="cuda").view(1, -1)
    kept = torch.sort(torch.where(slot < n, order, ld), dim=1)[0]
    live = slot < n
    idx = torch.where(live, kept, -1).to(torch.int32)
    b = torch.arange(B, device="cuda").view(-1, 1).expand(B, keep)[live]
    src, dst = kept[live], slot.expand(B, keep)[live]
    table = st["block_table"].long()
    a = table[b, src // BLK] * BLK + src % BLK
    z = table[b, dst // BLK] * BLK + dst % BLK
    for pool, width in (("kv_pool", D), ("k8_pool", 128), ("k_scale_pool", 1)):
        rows = st[pool].view(-1, width)
        rows[z] = rows[a]
    st["mass_out"][b, dst] = st["mass"][b, src]
    st["seq_len_out"].copy_(n.view(-1).clamp(max=keep))
    return idx, st["seq_len_out"], st["mass_out"], st["kv_pool"], st["k8_pool"], st["k_scale_pool"]


_PLAIN = dict(split=_plain_split, window=_plain_window, wdecode=_plain_wdecode, mass=_plain_mass,
              evict=_plain_evict)


# ------------------------------------------------------ the library's calls

def _workspace(st, nbytes):
    """The workspace a program keeps beside its cache."""
    if "ws" not in st:
        st["ws"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
    return st["ws"]


def _own(st):
    import sparse_attention_long_02_b200 as dsa
    op = st["op"]
    if op == "window":
        T, H = st["q"].shape[:2]
        ws = _workspace(st, dsa.window_mla_workspace_size(T, st["kv"].shape[0], H, st["q_pos0"],
                                                          st["sinks"], st["window"]))
        return dsa.window_mla(st["q"], st["kv"], st["sinks"], st["window"], SM_SCALE,
                              q_pos0=st["q_pos0"], workspace=ws)
    cache = (st["kv_pool"], st["block_table"], st["seq_len"])
    B, max_blocks = st["block_table"].shape
    if op == "split":
        ws = _workspace(st, dsa.split_mla_decode_workspace_size(B, st["nq"], max_blocks, st["H"]))
        return dsa.split_mla_decode_paged(st["q"], *cache, SM_SCALE, workspace=ws)
    if op == "wdecode":
        ws = _workspace(st, dsa.split_mla_decode_workspace_size(B, st["nq"], max_blocks, st["H"]))
        return dsa.window_mla_decode_paged(st["q"], *cache, st["sinks"], st["window"], SM_SCALE,
                                           workspace=ws)
    if op == "mass":
        return dsa.attention_mass_paged(st["q"], *cache, st["lse"], SM_SCALE, st["mass"])
    idx, lens, mass = dsa.cache_evict_paged(
        *cache, st["mass"], st["budget"], st["sinks"], st["recent"], k8_pool=st["k8_pool"],
        k_scale_pool=st["k_scale_pool"], seq_len_out=st["seq_len_out"], mass_out=st["mass_out"])
    return idx, lens, mass, st["kv_pool"], st["k8_pool"], st["k_scale_pool"]


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# -------------------------------------------------------------------- work

def _seen(qpos, sinks, window):
    if qpos < 0:
        return 0
    if not window or window > qpos:
        return qpos + 1
    return window + min(sinks, qpos - window + 1)


def work(case):
    op = case["op"]
    if op == "window":
        T, H, p0, s, w = (case[k] for k in ("T", "H", "q_pos0", "sinks", "window"))
        pairs = sum(_seen(p0 + t, s, w) for t in range(T))
        lo = max(0, p0 - w + 1)
        keys = p0 + T - lo + min(s, lo)
        return {"bytes": keys * D * 2 + T * H * (D * 2 + DV * 2 + 4),
                "flops": pairs * H * 2 * (D + DV)}
    lens = _lengths(case)
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        moved = sum(min(n, case["budget"]) for n in lens if n > case["budget"])
        # rows that have to move are read and written once; every total is read
        return {"bytes": moved * 2 * (D * 2 + 128 + 4) + 4 * sum(lens) + kept * 8, "flops": 0}
    nq, H = case["nq"], case["H"]
    s, w = case.get("sinks", 0), case.get("window", 0)
    pairs = sum(_seen(n - nq + j, s, w) for n in lens for j in range(nq))
    keys = sum(min(n, _seen(n - 1, s, w) + (nq - 1 if w else 0)) for n in lens)
    rows = len(lens) * nq * H
    if op == "mass":
        return {"bytes": keys * (D * 2 + 8) + rows * (D * 2 + 4), "flops": pairs * H * 2 * D}
    return {"bytes": keys * D * 2 + rows * (D * 2 + DV * 2 + 4), "flops": pairs * H * 2 * (D + DV)}


# ---------------------------------------------- the definitions in 64 bits

def _exact_row(q, k, see):
    """Softmax attention of queries q [r, 576] over keys k [n, 576], seen [r, n]."""
    z = (q.double() @ k.double().T) / math.sqrt(D)
    z = torch.where(see, z, torch.full_like(z, -math.inf))
    return z, torch.logsumexp(z, 1)


def _exact_seq(st, b, sinks, window):
    n, nq, H = int(st["seq_len"][b]), st["nq"], st["H"]
    blocks = st["block_table"][b, : (n + BLK - 1) // BLK].long()
    k = st["kv_pool"][blocks].reshape(-1, D)[:n]
    at = torch.arange(n, device="cuda")
    at_q = torch.arange(n - nq, n, device="cuda").repeat_interleave(H).unsqueeze(1)
    see = at <= at_q
    if window:
        see &= (at > at_q - window) | (at < sinks)
    return (*_exact_row(st["q"][b].reshape(nq * H, D), k, see), k)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("split", "wdecode"):
        outs, lses = [], []
        for b in range(case["B"]):
            z, lse, k = _exact_seq(st, b, case.get("sinks", 0), case.get("window", 0))
            p = torch.where(torch.isfinite(lse).unsqueeze(1), torch.exp(z - lse.unsqueeze(1)), 0.0)
            outs.append((p @ k[:, :DV].double()).view(case["nq"], case["H"], DV))
            lses.append(lse.view(case["nq"], case["H"]))
        return torch.stack(outs), torch.stack(lses)
    if op == "window":
        T, H, p0, s, w = (case[k] for k in ("T", "H", "q_pos0", "sinks", "window"))
        outs, lses = [], []
        for a in range(0, T, 256):
            e = min(T, a + 256)
            lo = max(0, p0 + a - w + 1)
            at = torch.cat([torch.arange(min(s, lo), device="cuda"),
                            torch.arange(lo, p0 + e, device="cuda")])
            k = st["kv"][at].double()
            at_q = torch.arange(p0 + a, p0 + e, device="cuda").repeat_interleave(H).unsqueeze(1)
            see = (at <= at_q) & ((at > at_q - w) | (at < s))
            z, lse = _exact_row(st["q"][a:e].reshape(-1, D), k, see)
            outs.append((torch.softmax(z, 1) @ k[:, :DV]).view(-1, H, DV))
            lses.append(lse.view(-1, H))
        return torch.cat(outs), torch.cat(lses)
    if op == "mass":
        mass = st["mass"].double()
        for b in range(case["B"]):
            z, _, _ = _exact_seq(st, b, 0, 0)
            n = z.shape[1]
            lse = st["lse"][b].reshape(-1, 1).double()
            got = torch.where(torch.isfinite(z), torch.exp(z - lse), 0.0).sum(0)
            mass[b, max(0, n - case["nq"]):n] = 0.0
            mass[b, :n] += got
        return mass
    idx = torch.full((case["B"], case["budget"]), -1, dtype=torch.int32)
    lens = st["seq_len"].cpu()
    new, mass = lens.clone(), st["mass"].cpu()
    out = st["mass_out"].double()
    pools = [st["kv_pool"].view(-1, D), st["k8_pool"].view(-1, 128), st["k_scale_pool"].view(-1, 1)]
    for b in range(case["B"]):
        n = int(lens[b])
        kept = list(range(n))
        if n > case["budget"]:
            free = range(case["sinks"], n - case["recent"])
            row = mass[b].tolist()
            best = sorted(free, key=lambda i: (-row[i], i))
            best = best[: case["budget"] - case["sinks"] - case["recent"]]
            kept = list(range(case["sinks"])) + sorted(best) + list(range(n - case["recent"], n))
        new[b] = len(kept)
        idx[b, : len(kept)] = torch.tensor(kept, dtype=torch.int32)
        src = torch.tensor(kept, dtype=torch.long, device="cuda")
        dst = torch.arange(len(kept), device="cuda")
        t = st["block_table"][b].long()
        for p in pools:
            p[t[dst // BLK] * BLK + dst % BLK] = p[t[src // BLK] * BLK + src % BLK].clone()
        out[b, : len(kept)] = st["mass"][b, src].double()
    return idx, new, out, st["kv_pool"], st["k8_pool"], st["k_scale_pool"]
