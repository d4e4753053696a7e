"""Measured cases of the paged key/value cache and of the attention that reads it.

Operators: attention of a few new tokens over a paged cache (``paged``), the same for a batch that
shares a long prefix (``shared``), growing sequences and writing their new keys and values
(``append``), and moving pages: forking sequences, copying pages, freeing sequences and compacting
the pool (``fork``, ``copy``, ``defrag``).

A cache is K, V [layers, pages, Hkv, page, d], a page table [slots, width] of page numbers (-1 behind
the last page of a sequence), the lengths [slots] and the number of tables that hold each page
[pages]. Each pass that changes the table, the lengths or the counts starts from a saved copy of
them, so passes repeat.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, kind, dtype="bf16", B=1, T=1, Hq=8, Hkv=8, d=128, page=16, layers=1, lo=1, hi=1,
          shared=0, window=-1, softcap=0.0, spread=1.0):
    return {"name": name, "kind": kind, "dtype": dtype, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv,
            "d": d, "page": page, "layers": layers, "lo": lo, "hi": hi, "shared": shared,
            "window": window, "softcap": softcap, "spread": spread}


def listed():
    return [
        # one user, a short dialogue, a small head size: nothing but latency
        _case("paged_one_short", "paged", B=1, Hq=12, Hkv=12, d=64, lo=211, hi=211),
        # a serving batch whose lengths span a factor of a thousand, grouped heads
        _case("paged_ragged", "paged", B=64, Hq=32, Hkv=8, lo=13, hi=16384),
        # five drafted tokens to check per sequence, a local window and capped scores, no grouping
        _case("paged_draft_window", "paged", B=16, T=5, Hq=32, Hkv=32, page=32, lo=500, hi=8190,
              window=2048, softcap=30.0),
        # four answers sampled from one short prompt, in fp32
        _case("shared_few_fp32", "shared", "f32", B=4, Hq=8, Hkv=2, d=32, lo=1, hi=40, shared=512),
        # a batch behind one system prompt
        _case("shared_prompt", "shared", B=64, Hq=32, Hkv=8, lo=1, hi=512, shared=4096),
        # a large batch of questions on one long document
        _case("shared_document", "shared", B=128, Hq=32, Hkv=8, page=64, lo=1, hi=2048,
              shared=16384),
        # one decoding step of a batch in four layers: latency, and a new page now and then
        _case("append_step", "append", B=48, T=1, Hkv=8, page=16, layers=4, lo=1, hi=4000),
        # a batch of ragged prompts in two layers: bandwidth
        _case("append_prompts", "append", B=24, T=4096, Hkv=8, page=64, layers=2, lo=0, hi=300,
              spread=200.0),
        # four samples forked from short prompts
        _case("fork_few", "fork", B=4, Hkv=12, d=64, page=16, layers=2, lo=90, hi=400),
        # one step of a search: 256 new beams forked from 64, the old ones freed, sixteen layers
        _case("fork_beams", "fork", B=64, T=4, Hkv=8, page=32, layers=16, lo=20, hi=2000),
        # a list of pages duplicated, eight layers
        _case("copy_pages", "copy", B=32, Hkv=8, page=16, layers=8, lo=100, hi=600),
        # every other sequence of a large pool ends, and the pages that live move to the front
        _case("defrag_pool", "defrag", B=128, Hkv=8, page=32, layers=8, lo=10, hi=1500),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    kind = rng.choice(["paged", "paged", "shared", "shared", "append", "fork", "copy", "defrag"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128] if dtype == "bf16" else [16, 32, 64, 128])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    size = {"bf16": 2, "f32": 4}[dtype]
    c = _case("", kind, dtype, Hkv=Hkv, d=d, page=page)
    if kind in ("paged", "shared"):
        c["B"] = _log(rng, 1, 128)
        c["T"] = rng.choice([1, 1, 1, 2, 3, 4, 8])
        # fp32 runs on the CUDA cores: fewer rows there
        c["Hq"] = Hkv * rng.choice([1, 2, 4, 5, 8] if dtype == "bf16" else [1, 2, 4])
        most = max(64, min(16384, 700_000_000 // (c["B"] * Hkv * d * size * 2)))
        c["hi"] = _log(rng, 20, most)
        c["lo"] = rng.choice([0, 1, max(1, c["hi"] // 3), c["hi"]])
        if rng.random() < 0.3:
            c["window"] = _log(rng, 8, 4096)
        if rng.random() < 0.25:
            c["softcap"] = rng.choice([20.0, 30.0, 50.0])
        if kind == "shared":
            c["B"] = max(2, c["B"])
            rows = c["B"] * c["T"] * c["Hq"] // Hkv
            top = 16384 if dtype == "bf16" else 4096
            c["hi"] = min(c["hi"], 2048)
            c["lo"] = min(c["lo"], c["hi"])
            c["shared"] = max(1, _log(rng, 100, min(top, max(400, 8_000_000 // rows))) // page) * page
    elif kind == "append":
        c["layers"] = rng.choice([1, 2, 4])
        c["B"] = _log(rng, 1, 64)
        c["T"] = rng.choice([1, 1, 5, 200, 2000])
        c["T"] = min(c["T"], 200_000_000 // (c["layers"] * c["B"] * Hkv * d * size * 2))
        c["spread"] = rng.choice([1.0, 1.0, 10.0, 100.0]) if c["T"] > 1 else 1.0
        c["hi"] = _log(rng, 10, 2000)
        c["lo"] = rng.choice([0, 1, c["hi"] // 2])
    else:
        c["layers"] = rng.choice([1, 2, 5, 8])
        c["B"] = _log(rng, 2, 128)
        if kind == "fork":
            c["T"] = rng.choice([1, 1, 2, 4])
            tail = c["T"] * c["layers"] * page * Hkv * d * size * 4
            c["B"] = max(2, min(c["B"], 64, 900_000_000 // tail))
        most = 1_000_000_000 // (c["layers"] * c["B"] * Hkv * d * size * 2)
        c["hi"] = _log(rng, 20, max(40, min(4000, most)))
        c["lo"] = rng.choice([1, max(1, c["hi"] // 2), c["hi"]])
    return c


def _spaced(n, lo, hi):
    """n whole numbers from lo to hi, even on a logarithmic scale (zero allowed)."""
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** ((i + 0.5) / n))) - 1 for i in range(n)]


def _counts(case):
    """New tokens of each sequence of an append case."""
    return _spaced(case["B"], max(1, int(case["T"] / case["spread"])), case["T"])


def _pairs(case):
    """Pages that a copy case duplicates: half of the first page count."""
    return max(1, sum(-(-n // case["page"]) for n in _lengths(case)) // 2)


def _lengths(case):
    """The lengths of a case's sequences, in the order of their sizes."""
    return [case["shared"] + n for n in _spaced(case["B"], case["lo"], case["hi"])]


def _fill(case, seed):
    """Tables, lengths, counts (host, int32) and sizes of a case's cache."""
    rng = np.random.default_rng(seed)
    B, page, kind = case["B"], case["page"], case["kind"]
    lens = rng.permutation(np.array(_lengths(case), dtype=np.int64))
    counts = rng.permutation(np.array(_counts(case), dtype=np.int64)) if kind == "append" else None
    copies = case["T"] if kind == "fork" else 0
    slots = B * (1 + copies) + 3
    # sizes follow from the case alone
    longest = case["shared"] + case["hi"] + (case["T"] if kind == "append" else 0)
    width = max(1, -(-longest // page)) + 1
    need = -(-lens // page)
    first = case["shared"] // page
    held = int(first + (need - first).sum())
    more = int((-(-counts // page)).sum()) + B if counts is not None else 0
    pages = held + more + B * copies + (_pairs(case) if kind == "copy" else 0) + 5
    order = rng.permutation(pages)
    slot = rng.permutation(slots)[:B]
    table = np.full((slots, width), -1, dtype=np.int32)
    refs = np.zeros(pages, dtype=np.int32)
    length = np.zeros(slots, dtype=np.int32)
    length[slot] = lens
    table[slot, :first] = order[:first]
    at = first
    for s, n in zip(slot, need):
        table[s, first:n] = order[at:at + n - first]
        at += n - first
    np.add.at(refs, table[table >= 0], 1)
    return table, length, refs, slot.astype(np.int32), counts, rng


def prepare(case, seed):
    table, length, refs, slot, counts, rng = _fill(case, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    B, T, Hkv, d, page, L = (case[n] for n in ("B", "T", "Hkv", "d", "page", "layers"))
    st = {"case": case, "k": normal(L, refs.size, Hkv, page, d),
          "v": normal(L, refs.size, Hkv, page, d)}
    # table, lengths and counts in one buffer, so that one copy brings them back
    saved = torch.from_numpy(np.concatenate([table.ravel(), length, refs])).cuda()
    meta = saved.clone()
    st["saved"], st["meta"] = saved, meta
    n, m = table.size, table.size + length.size
    st["table"], st["lens"], st["refs"] = meta[:n].view(table.shape), meta[n:m], meta[m:]
    st["seqs"] = torch.from_numpy(slot).cuda()
    kind = case["kind"]
    if kind in ("paged", "shared"):
        st["q"] = normal(B, case["Hq"], T, d)
    elif kind == "append":
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        st["cu"] = torch.from_numpy(cu).cuda()
        total = int(cu[-1])
        st["new_k"] = [normal(total, Hkv, d) for _ in range(L)]
        st["new_v"] = [normal(total, Hkv, d) for _ in range(L)]
        st["even"] = int(counts.max()) if counts.max() == counts.min() else 0
    elif kind == "fork":
        # children draw their parents freely; the parents are freed afterwards
        empty = np.setdiff1d(np.arange(length.size), slot)
        dst = rng.permutation(empty)[:B * T]
        src = slot[rng.integers(0, B, B * T)]
        st["src"], st["dst"] = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (src, dst))
    elif kind == "copy":
        free = np.flatnonzero(refs == 0)
        used = np.flatnonzero(refs)
        k = _pairs(case)
        st["src"] = torch.from_numpy(rng.choice(used, k).astype(np.int32)).cuda()
        st["dst"] = torch.from_numpy(rng.permutation(free)[:k].astype(np.int32)).cuda()
    elif kind == "defrag":
        st["done"] = torch.from_numpy(slot[:(B + 1) // 2].copy()).cuda()
    if own:
        from exact_io_aware_45_b200 import fa
        st["cache"] = fa.PagedCache(st["k"], st["v"], st["table"], st["lens"], st["refs"])
    return st


# ------------------------------------------------------------------ plain forms

def _attend(st, shared):
    """Scores, softmax and weighted sums over a dense copy of the keys and values that the table
    names, in 32 bits; the shared tokens are taken once."""
    case = st["case"]
    B, T, Hq, Hkv, d = (case[n] for n in ("B", "T", "Hq", "Hkv", "d"))
    G, page = Hq // Hkv, case["page"]
    rows = st["table"][st["seqs"].long()].long().clamp(min=0)
    length = st["lens"][st["seqs"].long()].long()
    width = rows.shape[1]
    first = shared // page

    def dense(x, pages):                      # [..., n] page numbers -> [..., Hkv, n * page, d]
        y = x[0][pages].float().transpose(-4, -3)
        return y.reshape(*y.shape[:-3], -1, d)

    q = st["q"].float().view(B, Hkv, G, T, d)
    k, v = (dense(st[n], rows[:, first:width]) for n in "kv")
    # what lies behind a sequence's end is not part of it
    at = torch.arange(first * page, width * page, device=q.device)
    gone = (at[None] >= length[:, None])[:, None, :, None]
    k, v = k.masked_fill(gone, 0.0), v.masked_fill(gone, 0.0)
    s = torch.einsum("bhgtd,bhnd->bhgtn", q, k)
    at = torch.arange(width * page, device=q.device)
    if shared:
        pk, pv = (dense(st[n], rows[0, :first]) for n in "kv")
        s = torch.cat([torch.einsum("bhgtd,hnd->bhgtn", q, pk), s], -1)
    s = s / math.sqrt(d)
    if case["softcap"]:
        s = case["softcap"] * torch.tanh(s / case["softcap"])
    spot = length[:, None] - T + torch.arange(T, device=q.device)          # [B, T]
    seen = (at <= spot[..., None]) & (at < length[:, None, None])
    if case["window"] >= 0:
        seen &= at >= spot[..., None] - case["window"]
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    z = p.sum(-1, keepdim=True)
    lse = (top + torch.log(z)).squeeze(-1)
    p = torch.where(z > 0, p / z, torch.zeros_like(p))
    n = first * page
    o = torch.einsum("bhgtn,bhnd->bhgtd", p[..., n:], v)
    if shared:
        o = o + torch.einsum("bhgtn,hnd->bhgtd", p[..., :n], pv)
    return o.to(st["q"].dtype).view(B, Hq, T, d), lse.view(B, Hq, T)


def _free_first(refs):
    """Page numbers with the free pages in front, lowest first."""
    return torch.sort((refs != 0).to(torch.int8), stable=True).indices


def _extend(st, counts):
    page, table, refs = st["case"]["page"], st["table"], st["refs"]
    seqs = st["seqs"].long()
    length = st["lens"][seqs].long()
    have, want = (-(-n // page) for n in (length, length + counts))
    before = torch.cumsum(want - have, 0) - (want - have)
    order = _free_first(refs)
    at = torch.arange(table.shape[1], device=refs.device)[None]
    fresh = (at >= have[:, None]) & (at < want[:, None])
    pick = (before[:, None] + at - have[:, None]).clamp(0, refs.numel() - 1)
    table[seqs] = torch.where(fresh, order[pick].int(), table[seqs])
    total = (want - have).sum()
    refs[order] = torch.where(torch.arange(refs.numel(), device=refs.device) < total,
                              torch.ones_like(refs), refs[order])
    st["lens"][seqs] = (length + counts).int()
    return length


def _append(st):
    case, cu = st["case"], st["cu"].long()
    seqs, page = st["seqs"].long(), case["page"]
    pos = _extend(st, cu[1:] - cu[:-1])
    total = st["new_k"][0].shape[0]
    row = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu, row, right=True) - 1
    at = pos[b] + row - cu[b]
    dst, off = st["table"][seqs[b], at // page].long(), at % page
    layer = torch.arange(case["layers"], device=cu.device)[:, None]
    st["k"][layer, dst, :, off] = torch.stack(st["new_k"])
    st["v"][layer, dst, :, off] = torch.stack(st["new_v"])
    return pos.int()


def _drop(st, seqs):
    """Frees sequences: each of their pages has one table less."""
    table, refs, seqs = st["table"], st["refs"], seqs.long()
    rows = table[seqs]
    refs.scatter_add_(0, rows.clamp(min=0).long().flatten(), -(rows >= 0).int().flatten())
    table[seqs] = -1
    st["lens"][seqs] = 0


def _fork(st):
    page, table, refs = st["case"]["page"], st["table"], st["refs"]
    src, dst = st["src"].long(), st["dst"].long()
    length = st["lens"][src].long()
    full, part = length // page, length % page > 0
    rows = table[src].long()
    at = torch.arange(table.shape[1], device=refs.device)[None]
    fresh = _free_first(refs)[(torch.cumsum(part, 0) - 1).clamp(min=0)]
    last = (at == full[:, None]) & part[:, None]
    child = torch.where(at < full[:, None], rows, torch.where(last, fresh[:, None], -1))
    old = torch.where(part, rows.gather(1, full[:, None])[:, 0], rows[:, 0])
    new = torch.where(part, fresh, old)
    refs.scatter_add_(0, child.clamp(min=0).flatten(), (child >= 0).int().flatten())
    table[dst] = child.int()
    st["lens"][dst] = length.int()
    st["k"][:, new] = st["k"][:, old]
    st["v"][:, new] = st["v"][:, old]
    _drop(st, st["seqs"])


def _copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    st["k"][:, dst] = st["k"][:, src]
    st["v"][:, dst] = st["v"][:, src]


def _defrag(st):
    _drop(st, st["done"])
    table, refs = st["table"], st["refs"]
    live = refs > 0
    at = torch.arange(refs.numel(), device=refs.device)
    front = at < live.sum()
    src, dst = torch.nonzero(live & ~front)[:, 0], torch.nonzero(~live & front)[:, 0]
    st["k"][:, dst] = st["k"][:, src]
    st["v"][:, dst] = st["v"][:, src]
    refs[dst] = refs[src]
    refs[src] = 0
    to = at.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    kind = case["kind"]
    if kind in ("paged", "shared"):
        if not own:
            return _attend(st, case["shared"])
        from exact_io_aware_45_b200 import fa
        more = dict(window_left=case["window"], softcap=case["softcap"])
        if kind == "paged":
            return fa.forward_paged(st["q"], st["cache"], 0, st["seqs"], **more)
        return fa.forward_shared(st["q"], st["cache"], 0, case["shared"], st["seqs"], **more)
    pos = None
    if kind != "copy":
        st["meta"].copy_(st["saved"])
    if kind == "append":
        if own:
            cu = None if st["even"] else st["cu"]
            pos = st["cache"].extend(st["seqs"], st["even"] or cu)
            for layer, (k, v) in enumerate(zip(st["new_k"], st["new_v"])):
                st["cache"].write(layer, k, v, st["seqs"], pos, cu)
        else:
            pos = _append(st)
    elif kind == "fork":
        if own:
            st["cache"].fork(st["src"], st["dst"])
            st["cache"].free(st["seqs"])
        else:
            _fork(st)
    elif kind == "copy":
        if own:
            st["cache"].copy_pages(st["src"], st["dst"])
        else:
            _copy(st)
    else:
        if own:
            st["cache"].free(st["done"])
            st["cache"].compact()
        else:
            _defrag(st)
    return {"k": st["k"], "v": st["v"], "table": st["table"], "lens": st["lens"],
            "refs": st["refs"], "pos": pos}


def work(case):
    size = {"bf16": 2, "f32": 4}[case["dtype"]]
    B, T, Hq, Hkv, d, page, L = (case[n] for n in ("B", "T", "Hq", "Hkv", "d", "page", "layers"))
    token = 2 * Hkv * d * size                      # K and V of one token in one layer
    kind, lens = case["kind"], _lengths(case)
    if kind in ("paged", "shared"):
        pairs, keys, lowest = 0, 0, case["shared"]
        for n in lens:
            lo = max(0, n - T - case["window"]) if case["window"] >= 0 else 0
            keys += n - max(lo, case["shared"])
            lowest = min(lowest, lo)
            for t in range(T):
                spot = n - T + t
                back = case["window"] if case["window"] >= 0 else spot
                pairs += max(0, min(spot, back) + 1)
        keys += case["shared"] - lowest
        tables = 4 * sum(-(-n // page) for n in lens)
        return {"bytes": keys * token + 2 * B * Hq * T * d * size + 4 * B * Hq * T + tables,
                "flops": 4.0 * d * Hq * pairs}
    held = sum(-(-n // page) for n in lens)
    meta = 4 * (held + B)
    if kind == "append":
        return {"bytes": 2 * sum(_counts(case)) * token * L + meta, "flops": 0}
    if kind == "fork":
        # each child's last page where it is not full, on the average of the parents
        part = sum(n % page > 0 for n in lens) * T
        return {"bytes": 2 * part * page * token * L + meta * (1 + 2 * T), "flops": 0}
    if kind == "copy":
        return {"bytes": 2 * _pairs(case) * (page * token * L + 4), "flops": 0}
    # the pages that live behind their count move, about half of the half that is left
    return {"bytes": 2 * (held // 4) * page * token * L + 3 * meta, "flops": 0}


# ------------------------------------------------------------------ definition in 64 bits

def exact(case, seed):
    """O and LSE of the attention cases, one sequence and KV head at a time, in 64 bits; the other
    cases move data and compute no numbers."""
    if case["kind"] not in ("paged", "shared"):
        return None
    st = prepare(case, seed)
    B, T, Hq, Hkv, d = (case[n] for n in ("B", "T", "Hq", "Hkv", "d"))
    G = Hq // Hkv
    o = torch.zeros(B, Hq, T, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    table, length, seqs = st["table"].cpu(), st["lens"].cpu().tolist(), st["seqs"].cpu().tolist()
    for b, s in enumerate(seqs):
        n = length[s]
        if n == 0:
            continue
        pages = table[s, :-(-n // case["page"])].long().cuda()
        k, v = (st[x][0, pages].permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n].double()
                for x in "kv")
        for t in range(T):
            hi = n - T + t
            lo = max(0, hi - case["window"]) if case["window"] >= 0 else 0
            if hi < 0:
                continue
            q = st["q"][b, :, t].double().view(Hkv, G, d)
            x = q @ k[:, lo:hi + 1].transpose(1, 2) * (float(d) ** -0.5)
            if case["softcap"]:
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            z = torch.logsumexp(x, -1, keepdim=True)
            o[b, :, t] = (torch.exp(x - z) @ v[:, lo:hi + 1]).view(Hq, d)
            lse[b, :, t] = z.view(Hq)
    return o, lse


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c, work(c))
