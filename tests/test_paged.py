"""Paged key/value cache (fa_cache_*) and attention over it (fa_fwd_paged, fa_fwd_shared).

CPU tests pin the oracle and check the argument handling of the C ABI; GPU tests compare the
kernels with the oracle.

Error bounds, before any run. With u = 2^-24 and the oracle's A = sum p |v| and X = scale max_j
sum |q||k|: a score is off by dx <= 2 (d + 8) u X (products and sums of d terms, where tensor cores
may truncate) plus 4e-7 cap under a soft cap; its exponential by 2^-21 besides; sums of n terms by n u.
So LSE is off by dx + (n + 64) u + 2^-20 (1 + |LSE|) and O by A (2 dx + 2 (n + 64) u + 2^-20) in fp32.
With bf16 the probabilities and the result are rounded: 2^-8 A and 2^-8 |O| more."""
import ctypes
import math

import numpy as np
import pytest

from exact_io_aware_45_b200 import fa
from oracle import paged as orc

U = 2.0 ** -24


# ------------------------------------------------------------------ oracle pins (CPU)

def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(4, 1, 8)), rng.normal(size=(2, 5, 8)), rng.normal(size=(2, 5, 8))
    O, L, A, X = orc.attend(q, k[:, :1], v[:, :1], 1, 0, 0.5)       # one key: O = V
    assert np.allclose(O[:, 0], v[[0, 0, 1, 1], 0]) and np.allclose(A, np.abs(O))
    assert np.allclose(L[:, 0], 0.5 * np.einsum("hd,hd->h", q[:, 0], k[[0, 0, 1, 1], 0]))
    O, L, _, _ = orc.attend(q, 0 * k, v, 1, 4, 0.5)                 # equal scores: the mean
    assert np.allclose(O[2, 0], v[1].mean(0)) and np.allclose(L, math.log(5))
    O, L, _, _ = orc.attend(q, k, v, 1, 4, 0.5, window_left=0)      # itself only
    assert np.allclose(O[0, 0], v[0, 4])
    O, L, _, _ = orc.attend(q, k, v, 1, -1, 0.5)                    # sees nothing
    assert not O.any() and np.all(np.isneginf(L))


def test_oracle_pool_keeps_its_counts():
    rng = np.random.default_rng(1)
    p = orc.Pool(40, 4, 12, 8)
    for _ in range(200):
        try:
            step(p, rng)
        except orc.Refused:
            pass
        held = p.table[p.table >= 0]
        assert np.array_equal(np.bincount(held, minlength=40), p.refs)
        assert np.array_equal((p.table >= 0).sum(1), -(-p.lens // 4))


def step(p, rng):
    """One random operation on a pool: (name, lists, what the oracle returns)."""
    seqs = p.lens.size
    kind = rng.choice(["extend", "extend", "fork", "fork", "free", "compact"])
    if kind == "extend":
        n = int(rng.integers(1, 5))
        s = rng.choice(seqs, n, replace=rng.random() < 0.1)
        c = rng.integers(0, 3 * p.ps, n)
        return kind, (s, c), p.extend(s, c)
    if kind == "fork":
        empty = np.flatnonzero(p.lens == 0)
        n = min(len(empty), int(rng.integers(1, 4)))
        dst = rng.choice(empty, n, replace=False) if n else np.array([0])
        src = rng.choice(np.flatnonzero(p.lens) if p.lens.any() else [0], len(dst))
        return kind, (src, dst), p.fork(src, dst)
    if kind == "free":
        s = rng.choice(seqs, 2, replace=rng.random() < 0.2)
        return kind, (s,), p.free(s)
    return kind, (), p.compact()


def test_oracle_compact_moves_into_the_holes_in_order():
    p = orc.Pool(8, 2, 3, 4)
    p.extend([0, 1, 2], [4, 2, 4])          # pages 0 1 | 2 | 3 4
    p.free([0])
    assert p.compact() == [(3, 0), (4, 1)]
    assert p.table[2].tolist() == [0, 1, -1, -1] and p.refs.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]


# ------------------------------------------------------------------ argument checks (CPU)

G = 0x10000    # never dereferenced: the checks fail or return before any launch


def view(**kw):
    a = dict(K=G, V=G, layer_stride=0, page_stride=2 * 16 * 64, layers=1, pages=10, Hkv=2,
             page_size=16, d=64, dtype=fa.FA_BF16, table=G, lens=G, refs=G, seqs=4, seq_pages=8,
             err=G)
    a.update(kw)
    return fa.FaCache(*(a[n] for n, _ in fa.FaCache._fields_))


def fwd(cache=None, shared=None, **kw):
    a = dict(layer=0, Q=G, O=G, LSE=G, seqs=G, B=2, T=1, Hq=4, scale=0.1, causal=1, wl=-1, cap=0.0,
             ws=G, wsb=1 << 40)
    a.update(kw)
    c = view() if cache is None else cache
    head = (ctypes.byref(c), a["layer"], a["Q"], a["O"], a["LSE"], a["seqs"], a["B"], a["T"],
            a["Hq"])
    tail = (a["scale"], a["causal"], a["wl"], a["cap"], a["ws"], a["wsb"], 0)
    return fa.fa_fwd_paged(*head, *tail) if shared is None else \
        fa.fa_fwd_shared(*head, shared, *tail)


BAD_CACHES = [
    (dict(K=0), fa.FA_ERR_INVALID_ARG), (dict(V=G + 8), fa.FA_ERR_INVALID_ARG),
    (dict(table=0), fa.FA_ERR_INVALID_ARG), (dict(refs=G + 2), fa.FA_ERR_INVALID_ARG),
    (dict(err=0), fa.FA_ERR_INVALID_ARG), (dict(pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=-1), fa.FA_ERR_INVALID_ARG), (dict(seq_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(dtype=3), fa.FA_ERR_INVALID_ARG), (dict(d=48), fa.FA_ERR_UNSUPPORTED),
    (dict(page_size=24), fa.FA_ERR_UNSUPPORTED), (dict(page_size=256), fa.FA_ERR_UNSUPPORTED),
    (dict(page_stride=2 * 16 * 64 - 8), fa.FA_ERR_INVALID_ARG),
    (dict(page_stride=2 * 16 * 64 + 4), fa.FA_ERR_INVALID_ARG),
    (dict(layers=2), fa.FA_ERR_INVALID_ARG),             # layers on top of each other
    (dict(layers=2, layer_stride=20484), fa.FA_ERR_INVALID_ARG),
    (dict(pages=1 << 30), fa.FA_ERR_UNSUPPORTED),
    (dict(seqs=1 << 20, seq_pages=1 << 20), fa.FA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches_are_refused(kw, want):
    c = view(**kw)
    r = ctypes.byref(c)
    assert fwd(c) == want and fwd(c, shared=16) == want
    assert fa.fa_cache_extend(r, G, 1, 0, 1, G, G, 1 << 40, 0) == want
    assert fa.fa_cache_write(r, 0, G, G, G, G, 1, 0, 1, 0) == want
    for fn in (fa.fa_cache_fork, fa.fa_cache_copy):
        assert fn(r, G, G, 1, G, 1 << 40, 0) == want
    assert fa.fa_cache_free(r, G, 1, G, 1 << 40, 0) == want
    assert fa.fa_cache_compact(r, G, 1 << 40, 0) == want
    assert fa.fa_cache_workspace_size(r, 1) == 0
    assert fa.fa_paged_workspace_size(r, 1, 1, 2, 0) == 0
    assert fa.fa_last_launch_count() == 0


@pytest.mark.parametrize("kw,want", [
    (dict(layer=1), fa.FA_ERR_INVALID_ARG), (dict(layer=-1), fa.FA_ERR_INVALID_ARG),
    (dict(Hq=3), fa.FA_ERR_INVALID_ARG), (dict(Hq=0), fa.FA_ERR_INVALID_ARG),
    (dict(B=-1), fa.FA_ERR_INVALID_ARG), (dict(T=-1), fa.FA_ERR_INVALID_ARG),
    (dict(B=5, seqs=0), fa.FA_ERR_INVALID_ARG),          # more sequences than slots
    (dict(causal=2), fa.FA_ERR_INVALID_ARG), (dict(wl=-2), fa.FA_ERR_INVALID_ARG),
    (dict(scale=math.nan), fa.FA_ERR_INVALID_ARG), (dict(cap=-1.0), fa.FA_ERR_INVALID_ARG),
    (dict(cap=math.inf), fa.FA_ERR_INVALID_ARG),
    (dict(Q=0), fa.FA_ERR_INVALID_ARG), (dict(O=G + 8), fa.FA_ERR_INVALID_ARG),
    (dict(LSE=0), fa.FA_ERR_INVALID_ARG), (dict(seqs=G + 1), fa.FA_ERR_INVALID_ARG),
    (dict(ws=0), fa.FA_ERR_INVALID_ARG), (dict(wsb=1000), fa.FA_ERR_INVALID_ARG),
    (dict(T=1 << 20), fa.FA_ERR_UNSUPPORTED), (dict(B=1 << 26, T=8), fa.FA_ERR_UNSUPPORTED),
    (dict(B=0, Q=0), fa.FA_OK), (dict(T=0, Q=0), fa.FA_OK),
])
def test_attention_argument_checks(kw, want):
    assert fwd(**kw) == want and fwd(shared=32, **kw) == want
    assert fa.fa_last_launch_count() == 0


@pytest.mark.parametrize("shared", [-16, 8, 17, 16 * 9])
def test_shared_is_whole_pages_of_a_table(shared):
    assert fwd(shared=shared) == fa.FA_ERR_INVALID_ARG


def test_list_argument_checks():
    c = view()
    r, big, bad = ctypes.byref(c), 1 << 40, fa.FA_ERR_INVALID_ARG
    assert fa.fa_cache_extend(r, 0, 1, 0, 1, G, G, big, 0) == bad
    assert fa.fa_cache_extend(r, G, 5, 0, 1, G, G, big, 0) == bad      # more than slots
    assert fa.fa_cache_extend(r, G, 1, 0, -1, G, G, big, 0) == bad
    assert fa.fa_cache_extend(r, G, 1, 0, 1, 0, G, big, 0) == bad
    assert fa.fa_cache_extend(r, G, 1, 0, 1, G, G, 100, 0) == bad
    assert fa.fa_cache_extend(r, G, 1, G + 2, 1, G, G, big, 0) == bad
    assert fa.fa_cache_extend(r, 0, 0, 0, 1, 0, 0, 0, 0) == fa.FA_OK
    assert fa.fa_cache_write(r, 1, G, G, G, G, 1, 0, 1, 0) == bad
    assert fa.fa_cache_write(r, 0, G, G, G, G, 2, 0, 3, 0) == bad      # uneven without offsets
    assert fa.fa_cache_write(r, 0, G + 4, G, G, G, 1, 0, 1, 0) == bad
    assert fa.fa_cache_write(r, 0, 0, 0, 0, 0, 0, 0, 0, 0) == fa.FA_OK
    for fn in (fa.fa_cache_fork, fa.fa_cache_copy):
        assert fn(r, G, 0, 1, G, big, 0) == bad
        assert fn(r, G, G, 11, G, big, 0) == bad
        assert fn(r, G, G, 1, 0, big, 0) == bad
        assert fn(r, 0, 0, 0, 0, 0, 0) == fa.FA_OK
    assert fa.fa_cache_free(r, G, -1, G, big, 0) == bad
    assert fa.fa_cache_compact(r, G + 4, big, 0) == bad
    assert fa.fa_last_launch_count() == 0


def test_new_status_has_a_name():
    assert fa.status_string(fa.FA_ERR_CACHE) == "FA_ERR_CACHE"


# ------------------------------------------------------------------ attention (GPU)

def build(lens, Hkv, d, page, dtype, layers=1, layout="plain", shared=0, seed=0, slack=3):
    """A cache holding sequences of the given lengths in scattered pages, all else NaN (which no
    result may show), and the dense keys and values per sequence [layers][Hkv, n, d]."""
    import torch
    rng = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    B = len(lens)
    width = max(1, -(-max(list(lens) + [shared]) // page)) + 1
    need = [max(0, -(-n // page) - shared // page) for n in lens]
    pages = shared // page + sum(need) + slack
    shape = (layers, pages, Hkv, page, d)
    if layout == "plain":
        k, v = (torch.full(shape, math.nan, dtype=dt, device="cuda") for _ in range(2))
    elif layout == "joined":            # K and V halves of one tensor
        kv = torch.full((layers, pages, 2, Hkv, page, d), math.nan, dtype=dt, device="cuda")
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:                               # layers inside the pages
        k, v = (torch.full((pages, layers, Hkv, page, d), math.nan, dtype=dt,
                           device="cuda").transpose(0, 1) for _ in range(2))
    order = rng.permutation(pages)
    slots = B + 2
    slot = rng.permutation(slots)[:B]
    table = np.full((slots, width), -1, dtype=np.int32)
    length = np.zeros(slots, dtype=np.int32)
    first, at = shared // page, shared // page
    # only the first sequence that reaches farthest into the shared pages names them
    reach = [min(n, shared) for n in lens]
    lead = reach.index(max(reach))
    held = -(-reach[lead] // page)
    table[slot[lead], :held] = order[:held]
    g = torch.Generator(device="cuda").manual_seed(seed)
    head = [torch.randn(layers, Hkv, shared, d, generator=g, device="cuda").to(dt)
            for _ in range(2)]
    dense = []
    for b, n in enumerate(lens):
        length[slot[b]] = n
        mine = order[at:at + need[b]]
        table[slot[b], first:first + need[b]] = mine
        at += need[b]
        own = [torch.randn(layers, Hkv, max(0, n - shared), d, generator=g, device="cuda").to(dt)
               for _ in range(2)]
        for x, y, z in zip((k, v), own, head):
            for j, p in enumerate(mine):
                part = y[:, :, j * page:(j + 1) * page]
                x[:, int(p), :, :part.shape[2]] = part
            if b == lead:
                top = max(lens)         # what no sequence is long enough to see stays NaN
                for j in range(first):
                    m = max(0, min(page, top - j * page))
                    x[:, int(order[j]), :, :m] = z[:, :, j * page:j * page + m]
        dense.append([torch.cat([z, y], 2)[:, :, :n] for z, y in zip(head, own)])
    refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    cache = fa.PagedCache(k, v, *(torch.from_numpy(x).cuda() for x in (table, length, refs)))
    return cache, torch.from_numpy(slot.astype(np.int32)).cuda(), dense


def check(o, lse, q, dense, lens, layer, dtype, scale, causal=True, wl=-1, cap=0.0):
    o, lse = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    B, Hq, T, d = o.shape
    for b in range(B):
        k, v = (x[layer].float().cpu().numpy() for x in dense[b])
        O, L, A, X = orc.attend(q[b].float().cpu().numpy(), k, v, T, lens[b] - T, scale, causal,
                                wl, cap)
        n = lens[b]
        dx = 2 * (d + 8) * U * X + 4e-7 * cap
        tol = A * (2 * dx + 2 * (n + 64) * U + 2.0 ** -20)[..., None]
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * (A + np.abs(O))
        gone = np.isneginf(L)
        assert np.array_equal(np.isneginf(lse[b]), gone), f"sequence {b}: rows that see nothing"
        assert not o[b][gone].any()
        off = np.abs(o[b] - O) - tol
        assert off.max() <= 0, f"sequence {b}: O off by {np.abs(o[b] - O).max():.3e}"
        ltol = dx + (n + 64) * U + 2.0 ** -20 * (1 + np.abs(np.where(gone, 0, L)))
        loff = np.abs(np.where(gone, 0, lse[b]) - np.where(gone, 0, L)) - ltol
        assert loff.max() <= 0, f"sequence {b}: LSE off by {loff.max():.3e} too much"


def attend_case(lens, Hq, Hkv, d, page, dtype, T=1, shared=0, layers=1, layer=0, layout="plain",
                causal=True, wl=-1, cap=0.0, scale=None, seed=0):
    import torch
    cache, seqs, dense = build(lens, Hkv, d, page, dtype, layers, layout, shared, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn(len(lens), Hq, T, d, generator=g, device="cuda").to(cache.dtype)
    scale = 1 / math.sqrt(d) if scale is None else scale
    kw = dict(scale=scale, causal=causal, window_left=wl, softcap=cap)
    if shared:
        o, lse = fa.forward_shared(q, cache, layer, shared, seqs, **kw)
    else:
        o, lse = fa.forward_paged(q, cache, layer, seqs, **kw)
    cache.check()
    check(o, lse, q, dense, lens, layer, dtype, scale, causal, wl, cap)
    return o, lse


TYPES = [("bf16", 128), ("bf16", 64), ("bf16", 32), ("bf16", 16), ("f32", 128), ("f32", 64),
         ("f32", 32), ("f32", 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_paged_lengths_round_pages(dtype, d, page):
    lens = [0, 1, 2, page - 1, page, page + 1, 2 * page - 1, 127, 128, 129, 300]
    attend_case(lens, 4, 2, d, page, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 12, 12), (1, 8, 1), (1, 10, 2), (2, 6, 2),
                                      (3, 16, 2), (7, 10, 2), (5, 32, 1), (33, 4, 1), (70, 6, 2)])
def test_paged_tokens_and_heads(dtype, d, T, Hq, Hkv):
    attend_case([0, 1, T - 1, T, 97, 260], Hq, Hkv, d, 16, dtype, T=T)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("wl,causal,cap", [(0, True, 0.0), (1, True, 0.0), (37, True, 0.0),
                                           (128, True, 20.0), (5, False, 0.0), (-1, False, 0.0),
                                           (-1, True, 5.0), (2147483647, True, 0.0)])
def test_paged_masks_and_softcap(dtype, d, wl, causal, cap):
    attend_case([3, 64, 200, 515, 0], 6, 2, d, 32, dtype, T=4, wl=wl, causal=causal, cap=cap)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("lens,Hq,Hkv,T", [([9001], 8, 2, 1), ([9001], 4, 4, 3),
                                           ([5000, 1, 0, 7, 3333], 16, 2, 1),
                                           ([700] * 9, 3, 3, 2), ([4096, 4097, 4095], 40, 1, 2)])
def test_paged_long_sequences_are_cut_and_joined(dtype, d, lens, Hq, Hkv, T):
    attend_case(lens, Hq, Hkv, d, 16, dtype, T=T)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(17, 4, 2), (40, 4, 2), (64, 2, 1), (129, 2, 2), (200, 4, 2)])
@pytest.mark.parametrize("wl,causal,cap,scale", [(-1, True, 0.0, None), (50, True, 0.0, None),
                                                 (300, False, 8.0, None), (-1, False, 0.0, -0.1),
                                                 (-1, True, 0.0, 0.0)])
def test_paged_chunks_of_tokens(d, T, Hq, Hkv, wl, causal, cap, scale):
    """Many rows per KV head, one and two query tiles of them and more."""
    attend_case([0, 1, T - 3, T, 260, 700], Hq, Hkv, d, 16, "bf16", T=T, wl=wl, causal=causal,
                cap=cap, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,T", [(3, 9), (12, 3), (40, 4)])
@pytest.mark.parametrize("wl,causal,cap,scale", [(100, True, 0.0, None), (-1, False, 8.0, None),
                                                 (40, True, 5.0, -0.2), (-1, True, 0.0, 0.0)])
def test_shared_rows_in_one_and_two_tiles(d, B, T, wl, causal, cap, scale):
    attend_case([128 + (31 * b) % 200 for b in range(B)], 8, 2, d, 64, "bf16", T=T, shared=128,
                wl=wl, causal=causal, cap=cap, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,G,wl,cap,causal", [(3, 8, -1, 0.0, True), (4, 5, 30, 0.0, True),
                                               (17, 1, -1, 20.0, False), (23, 1, 5, 10.0, True)])
def test_paged_row_tiles_of_24(d, T, G, wl, cap, causal):
    """17 to 24 rows with many heads in the batch, with few, and behind a prefix."""
    lens = [0, 1, 16, 17, 100, 255, 256, 700, 33, 1500]
    attend_case(lens, 4 * G, 4, d, 16, "bf16", T=T, wl=wl, cap=cap, causal=causal)
    attend_case(lens[4:7], 2 * G, 2, d, 64, "bf16", T=T, wl=wl, cap=cap, causal=causal)
    attend_case([64 + n for n in lens], 4 * G, 4, d, 32, "bf16", T=T, shared=64, wl=wl, cap=cap,
                causal=causal)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,G", [(4, 8), (29, 1), (5, 5)])
@pytest.mark.parametrize("longest", [900, 2500])
def test_paged_two_row_tiles(d, T, G, longest):
    """25 to 32 rows, over tables for short and for long sequences, alone and behind a prefix."""
    lens = [0, 1, 31, 128, 129, 500, longest]
    attend_case(lens, 2 * G, 2, d, 16, "bf16", T=T, wl=200)
    attend_case([640 + n for n in lens], 2 * G, 2, d, 128, "bf16", T=T, shared=640, cap=25.0)
    attend_case([1280, 1300], 2 * G, 2, d, 64, "bf16", T=T, shared=1280)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,G", [(8, 5), (8, 8), (33, 1), (12, 4), (13, 5)])
@pytest.mark.parametrize("B", [3, 40])
def test_paged_many_rows_of_short_sequences(d, T, G, B):
    """33 to 65 rows where no table can hold more than 256 keys, alone and behind a prefix."""
    lens = [(13 * b * b + 7 * b) % 200 for b in range(B)]
    attend_case(lens, G, 1, d, 16, "bf16", T=T, wl=50, cap=25.0)
    attend_case([128 + n for n in lens], 2 * G, 2, d, 32, "bf16", T=T, shared=128)


CUDA_CORES = [("f32", 128), ("f32", 64), ("f32", 32), ("f32", 16), ("bf16", 32), ("bf16", 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", CUDA_CORES)
@pytest.mark.parametrize("T,G", [(1, 2), (3, 1), (4, 1), (5, 1), (1, 16), (17, 1), (16, 4), (13, 5),
                                 (50, 3)])
def test_paged_rows_on_the_cuda_cores(dtype, d, T, G):
    """One to four rows, part of a tile of 64, one tile, several; masks that leave rows empty."""
    lens = [0, 1, 15, 31, 32, 33, 100, 401]
    attend_case(lens, 2 * G, 2, d, 16, dtype, T=T)
    attend_case(lens, 2 * G, 2, d, 32, dtype, T=T, wl=20, cap=15.0, layers=2, layer=1,
                layout="joined")
    attend_case(lens, 2 * G, 2, d, 128, dtype, T=T, wl=7, causal=False, scale=-0.3, layout="inside")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", CUDA_CORES)
@pytest.mark.parametrize("B,T,shared", [(3, 1, 64), (16, 1, 480), (17, 4, 160), (70, 1, 1024)])
def test_shared_rows_on_the_cuda_cores(dtype, d, B, T, shared):
    lens = [shared - 20 + (11 * b * b) % 150 for b in range(B)]
    attend_case(lens, 4, 1, d, 32, dtype, T=T, shared=shared)
    attend_case(lens, 4, 1, d, 32, dtype, T=T, shared=shared, wl=shared - 40, cap=20.0)


@pytest.mark.gpu
def test_paged_many_sequences():
    """More sequences than threads of a block that scans their lengths."""
    rng = np.random.default_rng(3)
    attend_case([int(x) for x in rng.integers(0, 40, 700)], 2, 1, 64, 16, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["joined", "layers inside"])
def test_paged_strided_caches_and_layers(dtype, layout):
    for layer in (0, 2):
        attend_case([50, 17, 133], 8, 2, 64, 16, dtype, layers=3, layer=layer, layout=layout)
        attend_case([50, 97, 133], 8, 2, 64, 16, dtype, layers=3, layer=layer, layout=layout,
                    shared=48)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_paged_scales(scale):
    attend_case([5, 64, 200], 4, 2, 64, 16, "bf16", T=2, scale=scale)
    attend_case([5, 64, 200], 4, 2, 64, 16, "bf16", T=2, scale=scale, shared=32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 64)])
@pytest.mark.parametrize("shared,page", [(16, 16), (112, 16), (128, 128), (416, 32)])
@pytest.mark.parametrize("B,Hq,Hkv,T", [(1, 4, 2, 1), (5, 4, 4, 1), (9, 8, 1, 2), (40, 8, 2, 1),
                                        (3, 24, 2, 7)])
def test_shared_prefix(dtype, d, shared, page, B, Hq, Hkv, T):
    lens = [shared + (7 * b * b) % 90 for b in range(B)]
    attend_case(lens, Hq, Hkv, d, page, dtype, T=T, shared=shared)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("wl,cap,causal", [(10, 0.0, True), (100, 30.0, True), (300, 0.0, False),
                                           (-1, 20.0, False)])
def test_shared_masks(dtype, d, wl, cap, causal):
    """Windows that end inside the prefix for some sequences, sequences shorter than it."""
    lens = [0, 3, 100, 255, 256, 257, 300, 700] + [256 + 5 * i for i in range(20)]
    attend_case(lens, 8, 2, d, 32, dtype, T=3, shared=256, wl=wl, cap=cap, causal=causal)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 32)])
def test_shared_prefix_longer_than_every_sequence(dtype, d):
    """What no sequence is long enough to see of it holds NaN."""
    attend_case([90, 0, 17, 3], 8, 2, d, 32, dtype, T=2, shared=256)
    attend_case([0, 0], 8, 2, d, 32, dtype, shared=64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,reps", [("bf16", 128, 1), ("bf16", 64, 9), ("f32", 64, 2)])
def test_shared_padding_stands_anywhere(dtype, d, reps):
    """Slots out of range and an empty one before, between and behind the sequences."""
    import torch
    lens = [0, 40, 300, 256, 511] * reps
    cache, seqs, dense = build(lens, 2, d, 32, dtype, shared=256)
    order = [-1, 0, 1, None, 2, 3, None, 4]             # None: out of range; -1 as well
    order = [o if o is None or o < 0 else o + 5 * i for i in range(reps) for o in order]
    slots = torch.tensor([-1 if o == -1 else 10 ** 6 if o is None else int(seqs[o])
                          for o in order], dtype=torch.int32, device="cuda")
    real = [i for i, o in enumerate(order) if o is not None and o >= 0]
    q = torch.randn(len(order), 8, 3, d, device="cuda").to(cache.dtype)
    o, lse = fa.forward_shared(q, cache, 0, 256, slots)
    cache.check()
    check(o[real], lse[real], q[real], dense, lens, 0, dtype, d ** -0.5)
    pad = [i for i in range(len(order)) if i not in real]
    assert not o[pad].any() and torch.isneginf(lse[pad]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_shared_long_prefix(dtype, d):
    attend_case([4096 + 100 * i for i in range(6)], 8, 2, d, 64, dtype, shared=4096)
    attend_case([4096 + i for i in range(33)], 16, 2, d, 16, dtype, shared=4096)


@pytest.mark.gpu
def test_shared_equals_paged_on_forks():
    """The same tables with and without the promise of a shared prefix."""
    import torch
    cache = fa.PagedCache.new(2, 200, 2, 16, 64, 40, 20)
    seqs = torch.arange(33, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(133, 2, 64, device="cuda").bfloat16() for _ in range(2))
    pos = cache.extend(seqs[:1], 133)
    cache.write(1, k, v, seqs[:1], pos)
    cache.fork(seqs[:1].expand(32).contiguous(), seqs[1:])
    pos = cache.extend(seqs, 9)
    k, v = (torch.randn(33 * 9, 2, 64, device="cuda").bfloat16() for _ in range(2))
    cache.write(1, k, v, seqs, pos)
    cache.check()
    q = torch.randn(33, 8, 9, 64, device="cuda").bfloat16()
    o, lse = fa.forward_paged(q, cache, 1, seqs)
    for shared in (16, 128):
        o2, lse2 = fa.forward_shared(q, cache, 1, shared, seqs)
        # either is off by 2^-8 (A + |O|) and sum p |v| <= max |v|
        assert (o.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * v.float().abs().max()
        assert (lse - lse2).abs().max() <= 2e-5


@pytest.mark.gpu
def test_paged_slots_out_of_range_see_nothing():
    import torch
    cache, seqs, dense = build([20, 30], 2, 64, 16, "bf16")
    q = torch.randn(4, 2, 1, 64, device="cuda").bfloat16()
    odd = torch.tensor([int(seqs[0]), -1, 99, int(seqs[1])], dtype=torch.int32, device="cuda")
    o, lse = fa.forward_paged(q, cache, 0, odd)
    check(o[[0, 3]], lse[[0, 3]], q[[0, 3]], dense, [20, 30], 0, "bf16", 0.125)
    assert not o[1:3].any() and torch.isneginf(lse[1:3]).all()


@pytest.mark.gpu
def test_paged_default_slots_and_given_buffers():
    import torch
    cache, _, _ = build([20, 30, 40], 2, 64, 16, "bf16")
    q = torch.randn(5, 2, 1, 64, device="cuda").bfloat16()
    o, lse = fa.forward_paged(q, cache, 0)
    every = torch.arange(5, dtype=torch.int32, device="cuda")
    out, l2 = torch.empty_like(o), torch.empty_like(lse)
    ws = torch.empty(fa.fa_paged_workspace_size(cache._ref, 5, 1, 2, 0), dtype=torch.uint8,
                     device="cuda")
    r = fa.forward_paged(q, cache, 0, every, out=out, lse=l2, workspace=ws)
    assert r[0] is out and torch.equal(o, out) and torch.equal(lse, l2)


@pytest.mark.gpu
def test_paged_refusals_in_python():
    import torch
    cache, seqs, _ = build([20, 30], 2, 64, 16, "bf16")
    q = torch.randn(2, 4, 1, 64, device="cuda").bfloat16()
    for bad in (q.float(), q[:, :, :, :32], q.transpose(1, 2), q.cpu()):
        with pytest.raises((ValueError, fa.FaError)):
            fa.forward_paged(bad, cache, 0, seqs)
    for s in (seqs[:1], seqs.long(), seqs.cpu()):
        with pytest.raises(ValueError):
            fa.forward_paged(q, cache, 0, s)
    with pytest.raises(fa.FaError):
        fa.forward_paged(q, cache, 1, seqs)
    with pytest.raises(fa.FaError):
        fa.forward_shared(q, cache, 0, 8, seqs)
    with pytest.raises(ValueError):
        fa.forward_paged(q, cache, 0, seqs, out=torch.empty(2, 4, 1, 32, device="cuda"))
    with pytest.raises(ValueError):
        cache.extend(seqs, seqs)
    with pytest.raises(ValueError):
        cache.write(0, q[:, 0], q[:, 0], seqs, seqs)
    with pytest.raises(ValueError):
        cache.fork(seqs, seqs[:1])


# ------------------------------------------------------------------ pages (GPU)

def ints(x):
    import torch
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def same_state(cache, pool):
    for got, want in zip((cache.table, cache.lens, cache.refs), pool.state()):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("pages,seqs,dtype", [(40, 12, "f32"), (700, 30, "bf16"),
                                              (5000, 600, "bf16"), (20000, 300, "bf16")])
def test_pages_follow_the_oracle(pages, seqs, dtype):
    """A long run of operations; K and V stay with their tokens."""
    import torch
    rng = np.random.default_rng(pages)
    ps = 16
    pool = orc.Pool(pages, ps, seqs, 8)
    cache = fa.PagedCache.new(2, pages, 1, ps, 16, seqs, 8,
                              torch.float32 if dtype == "f32" else torch.bfloat16)
    k, v = (np.zeros((2, pages, ps, 16), dtype=np.float32) for _ in range(2))
    for _ in range(60):
        try:
            if rng.random() < 0.5 and pages > 100:      # a large extension
                n = int(rng.integers(1, seqs))
                s, c = rng.permutation(seqs)[:n], rng.integers(0, 30, n)
                what, lists, got = "extend", (s, c), pool.extend(s, c)
            else:
                what, lists, got = step(pool, rng)
        except orc.Refused:
            continue                                    # the pool is as it was
        if what == "extend":
            cu = np.concatenate([[0], np.cumsum(lists[1])])
            pos = cache.extend(ints(lists[0]), ints(cu))
            assert np.array_equal(pos.cpu().numpy(), got)
            total = int(cu[-1])
            if total:
                nk, nv = (torch.randn(2, total, 1, 16, device="cuda").to(cache.dtype)
                          for _ in range(2))
                for layer in range(2):
                    cache.write(layer, nk[layer], nv[layer], ints(lists[0]), pos, ints(cu))
                for i, s in enumerate(lists[0]):
                    for j in range(int(lists[1][i])):
                        p, r = pool.where(s, int(got[i]) + j)
                        k[:, p, r] = nk[:, cu[i] + j, 0].float().cpu().numpy()
                        v[:, p, r] = nv[:, cu[i] + j, 0].float().cpu().numpy()
        else:
            getattr(cache, what)(*map(ints, lists))
            for a, b in got or []:
                k[:, b], v[:, b] = k[:, a], v[:, a]
        same_state(cache, pool)
        cache.check()
    for x, y in ((cache.k, k), (cache.v, v)):
        assert np.array_equal(x[:, :, 0].float().cpu().numpy(), y)


@pytest.mark.gpu
def test_refused_page_calls_change_nothing():
    import torch
    cache = fa.PagedCache.new(1, 12, 2, 16, 32, 6, 4, torch.float32)
    pool = orc.Pool(12, 16, 6, 4)
    cache.extend(ints([0, 2]), ints([0, 40, 57]))
    pool.extend([0, 2], [40, 17])
    cache.k.normal_(), cache.v.normal_()
    k, v = cache.k.clone(), cache.v.clone()
    calls = [
        lambda: cache.extend(ints([1, 1]), 4),           # twice the same slot
        lambda: cache.extend(ints([1, 6]), 4),           # no such slot
        lambda: cache.extend(ints([-1]), 4),
        lambda: cache.extend(ints([0]), 25),             # longer than a table
        lambda: cache.extend(ints([1, 3, 4]), 40),       # nine pages, seven free
        lambda: cache.extend(ints([1, 3]), ints([0, 4, 2])),
        lambda: cache.fork(ints([0]), ints([2])),        # in use
        lambda: cache.fork(ints([0, 0]), ints([3, 3])),
        lambda: cache.fork(ints([0, 3]), ints([3, 4])),  # a source that is a destination
        lambda: cache.fork(ints([7]), ints([3])),
        lambda: cache.fork(ints([0]), ints([-3])),
        lambda: cache.free(ints([0, 0])),
        lambda: cache.free(ints([0, 9])),
        lambda: cache.copy_pages(ints([0, 1]), ints([5, 5])),
        lambda: cache.copy_pages(ints([0, 5]), ints([5, 6])),
        lambda: cache.copy_pages(ints([0]), ints([0])),
        lambda: cache.copy_pages(ints([0]), ints([12])),
        lambda: cache.copy_pages(ints([-1]), ints([7])),
    ]
    for call in calls:
        pos = call()
        with pytest.raises(fa.FaError) as e:
            cache.check()
        assert e.value.status == fa.FA_ERR_CACHE
        cache.check()                                    # read and cleared
        same_state(cache, pool)
        assert torch.equal(cache.k, k) and torch.equal(cache.v, v)
        if pos is not None:
            assert (pos == -1).all()
            new = torch.ones(2 * len(pos), 2, 32, device="cuda")
            cache.write(0, new, new, ints(np.zeros(len(pos))), pos)     # skipped
            cache.check()
            assert torch.equal(cache.k, k)


@pytest.mark.gpu
def test_write_refuses_what_is_shared_or_behind_the_end():
    import torch
    cache = fa.PagedCache.new(1, 12, 1, 16, 32, 4, 4, torch.float32)
    cache.extend(ints([0]), 20)
    cache.fork(ints([0]), ints([1]))
    new = torch.ones(20, 1, 32, device="cuda")
    cache.write(0, new, new, ints([0]), ints([10]))      # 10..15 shared, 16..19 its own, then the end
    with pytest.raises(fa.FaError):
        cache.check()
    k = cache.k[0, :, 0, :, 0].cpu().numpy()
    rows = cache.table.cpu().numpy()
    assert k[rows[0, 1], :4].tolist() == [1, 1, 1, 1] and k.sum() == 4
    cache.write(0, new[:1], new[:1], ints([9]), ints([0]))
    with pytest.raises(fa.FaError):
        cache.check()
    assert cache.k.sum() == 4 * 32


@pytest.mark.gpu
@pytest.mark.parametrize("page,Hkv,d,dtype", [(16, 1, 16, "bf16"), (128, 3, 128, "f32"),
                                              (32, 8, 64, "bf16")])
@pytest.mark.parametrize("layout", ["plain", "joined", "layers inside"])
def test_copy_pages(page, Hkv, d, dtype, layout):
    import torch
    cache, _, _ = build([9 * page], Hkv, d, page, dtype, layers=3, layout=layout, slack=9)
    cache.k.normal_(), cache.v.normal_()
    k, v = cache.k.clone(), cache.v.clone()
    src, dst = [3, 3, 0, 7, 11], [5, 12, 17, 1, 2]
    cache.copy_pages(ints(src), ints(dst))
    cache.check()
    k[:, dst], v[:, dst] = k[:, src], v[:, src]
    assert torch.equal(cache.k, k) and torch.equal(cache.v, v)


@pytest.mark.gpu
def test_copy_of_many_pages_and_its_refusal():
    import torch
    cache = fa.PagedCache.new(1, 20000, 1, 16, 16, 2, 2)
    cache.k.normal_(), cache.v.normal_()
    k = cache.k.clone()
    order = np.random.default_rng(0).permutation(20000)
    src, dst = order[:9500], order[9500:19000]
    cache.copy_pages(ints(src), ints(dst))
    cache.check()
    k[:, torch.from_numpy(dst).cuda()] = k[:, torch.from_numpy(src).cuda()]
    assert torch.equal(cache.k, k)
    dst[-1] = src[0]
    cache.copy_pages(ints(src[::-1].copy()), ints(dst))
    with pytest.raises(fa.FaError):
        cache.check()
    assert torch.equal(cache.k, k)


@pytest.mark.gpu
def test_extension_by_more_than_there_is():
    """Needs that add up past 32 bits are refused like others."""
    n = 900
    cache = fa.PagedCache.new(1, 20, 1, 128, 16, n, 2000000)
    cache.extend(ints(np.arange(n)), 250_000_000)
    with pytest.raises(fa.FaError):
        cache.check()
    assert not cache.lens.any() and not cache.refs.any()


@pytest.mark.gpu
def test_calls_on_a_side_stream():
    """A whole step on a stream of its own, its inputs made there; nothing waits for another."""
    import torch
    res = []
    for side in (False, True):
        s = torch.cuda.Stream() if side else torch.cuda.current_stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g = torch.Generator(device="cuda").manual_seed(1)
            cache = fa.PagedCache.new(1, 300, 2, 16, 64, 40, 40)
            slots = ints(np.arange(30))
            for n in (100, 1, 1):
                pos = cache.extend(slots, n)
                k, v = (torch.randn(30 * n, 2, 64, generator=g, device="cuda").bfloat16()
                        for _ in range(2))
                cache.write(0, k, v, slots, pos)
            q = torch.randn(30, 8, 1, 64, generator=g, device="cuda").bfloat16()
            r = fa.forward_paged(q, cache, 0, slots)
            cache.check()
        res.append([x.clone() for x in r])
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*res))


# ------------------------------------------------------------------ together (GPU)

def dense_of(log, slot, layer):
    import torch
    return [torch.cat([x[i] for x in log[slot][layer]], 1) for i in range(2)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 32)])
def test_a_serving_run(dtype, d):
    """A prompt, forks of it, steps behind the shared prefix, a fork of a fork, sequences that
    end, compaction, and steps again; each attention against the oracle."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    L, Hkv, Hq, page = 2, 2, 8, 16
    cache = fa.PagedCache.new(L, 64, Hkv, page, d, 10, 12, dt)
    log = {}
    gen = torch.Generator(device="cuda").manual_seed(7)

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda").to(dt)

    def grow(slots, counts, shared):
        cu = np.concatenate([[0], np.cumsum(counts)])
        even = len(set(counts)) == 1
        pos = cache.extend(ints(slots), counts[0] if even else ints(cu))
        for layer in range(L):
            k, v = randn(int(cu[-1]), Hkv, d), randn(int(cu[-1]), Hkv, d)
            cache.write(layer, k, v, ints(slots), pos, None if even else ints(cu))
            for i, s in enumerate(slots):
                part = [x[cu[i]:cu[i + 1]].transpose(0, 1) for x in (k, v)]
                log.setdefault(s, [[] for _ in range(L)])[layer].append(part)
            q = randn(len(slots), Hq, counts[0], d)
            o, lse = (fa.forward_shared(q, cache, layer, shared, ints(slots)) if shared else
                      fa.forward_paged(q, cache, layer, ints(slots)))
            lens = cache.lens.cpu().numpy()
            check(o, lse, q, [[x[None] for x in dense_of(log, s, layer)] for s in slots],
                  [int(lens[s]) for s in slots], 0, dtype, 1 / math.sqrt(d))
        cache.check()

    def fork(src, dst):
        cache.fork(ints(src), ints(dst))
        for a, b in zip(src, dst):
            log[b] = [list(x) for x in log[a]]

    grow([3], [69], 0)
    grow([5, 6], [30, 7], 0)
    fork([3, 3, 3], [0, 1, 2])
    for _ in range(3):
        grow([3, 0, 1, 2], [1] * 4, 64)
    fork([1, 5], [7, 8])
    grow([3, 0, 1, 2, 7], [5] * 5, 64)
    cache.free(ints([5, 3, 0]))
    cache.compact()
    cache.check()
    assert int((cache.refs > 0).sum()) == int(cache.refs.nonzero().max()) + 1
    grow([1, 2, 7], [12] * 3, 64)
    grow([8, 6], [3, 3], 0)


@pytest.mark.gpu
def test_a_captured_step_replays():
    """Two graphs of one decoding step each (extend, write, attend), replayed in turn and at once
    on two streams, on two caches: their workspaces are their own."""
    import torch
    res = []
    for graphs in (False, True):
        torch.manual_seed(3)
        work = []
        for i in range(2):
            cache = fa.PagedCache.new(1, 80, 2, 16, 64, 4, 20)
            seqs = ints([2, 0, 3])
            pos = cache.extend(seqs, 130 + i)
            k, v = (torch.randn(3 * (130 + i), 2, 64, device="cuda").bfloat16() for _ in range(2))
            cache.write(0, k, v, seqs, pos)
            k, v, q = (torch.randn(*s, device="cuda").bfloat16() for s in
                       ((3, 2, 64), (3, 2, 64), (3, 8, 1, 64)))
            o = torch.empty_like(q)

            def one(cache=cache, seqs=seqs, k=k, v=v, q=q, o=o):
                pos = cache.extend(seqs, 1)
                cache.write(0, k, v, seqs, pos)
                fa.forward_paged(q, cache, 0, seqs, out=o)

            work.append((cache, one, o))
        torch.cuda.synchronize()
        if graphs:
            made = []
            for cache, one, o in work:
                keep = [x.clone() for x in (cache.table, cache.lens, cache.refs)]
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    one()
                torch.cuda.synchronize()
                for x, y in zip((cache.table, cache.lens, cache.refs), keep):
                    assert torch.equal(x, y)
                made.append(g)
            streams = [torch.cuda.Stream() for _ in made]
            for _ in range(20):
                for g, s in zip(made, streams):
                    with torch.cuda.stream(s):
                        g.replay()
        else:
            for _ in range(20):
                for _, one, _ in work:
                    one()
        torch.cuda.synchronize()
        for cache, _, o in work:
            cache.check()
            res.append((o.clone(), cache.table.clone(), cache.lens.clone(), cache.k.clone()))
    for a, b in zip(res[:2], res[2:]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_paged_results_repeat_bit_for_bit():
    import torch
    cache, seqs, _ = build([3000, 1, 700, 4096], 2, 128, 16, "bf16")
    q = torch.randn(4, 8, 2, 128, device="cuda").bfloat16()
    first = fa.forward_paged(q, cache, 0, seqs)
    for _ in range(20):
        again = fa.forward_paged(q, cache, 0, seqs)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.gpu
def test_paged_large_offsets():
    """A cache of more than 2^31 elements: pages at both ends of it."""
    import torch
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB free")
    pages = (1 << 31) // (8 * 128 * 128) + 40
    cache = fa.PagedCache.new(1, pages, 8, 128, 128, 2, 4)
    n = 300
    x = [torch.randn(1, 8, n, 128, device="cuda").bfloat16() for _ in range(2)]
    rows = [pages - 1, 3, pages - 7, -1]
    for t, y in zip((cache.k, cache.v), x):
        for j in range(3):
            part = y[0, :, j * 128:(j + 1) * 128]
            t[0, rows[j], :, :part.shape[1]] = part
    cache.table[1] = ints(rows)
    cache.lens[1] = n
    cache.refs[[pages - 1, 3, pages - 7]] = 1
    q = torch.randn(1, 16, 1, 128, device="cuda").bfloat16()
    for shared in (0, 256):
        o, lse = (fa.forward_shared(q, cache, 0, shared, ints([1])) if shared else
                  fa.forward_paged(q, cache, 0, ints([1])))
        check(o, lse, q, [x], [n], 0, "bf16", 1 / math.sqrt(128))
    cache.compact()
    cache.check()
    assert cache.table[1].tolist() == [2, 0, 1, -1]     # 3, pages - 7 and pages - 1, in order
    o2, lse2 = fa.forward_paged(q, cache, 0, ints([1]))
    check(o2, lse2, q, [x], [n], 0, "bf16", 1 / math.sqrt(128))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shared,B,T", [(0, 3, 9), (0, 2, 70), (64, 12, 1), (64, 90, 2)])
def test_a_wait_that_runs_out_is_reported(d, shared, B, T):
    """The injected wait ends the call without a fault; err says so, and later calls work."""
    import time

    import torch
    lens = [400 + b for b in range(B)]
    cache, seqs, dense = build(lens, 2, d, 16, "bf16", shared=shared)
    q = torch.randn(B, 8, T, d, device="cuda").bfloat16()

    def call():
        return (fa.forward_shared(q, cache, 0, shared, seqs) if shared else
                fa.forward_paged(q, cache, 0, seqs))

    call()
    torch.cuda.synchronize()
    assert fa.fa_debug_set_stall(fa.FA_STALL_FWD, 4_000_000) == fa.FA_OK
    try:
        t0 = time.time()
        call()
        torch.cuda.synchronize()
        assert time.time() - t0 < 2
    finally:
        fa.fa_debug_set_stall(0, 0)
    call()                               # leaves at once: the word is set
    with pytest.raises(fa.FaError) as e:
        cache.check()
    assert e.value.status == fa.FA_ERR_TIMEOUT
    cache.check()
    o, lse = call()
    check(o, lse, q, dense, lens, 0, "bf16", 1 / math.sqrt(d))
