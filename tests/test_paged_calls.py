"""Calls of the paged cache and its attention at the edges of what include/fa.h allows: empty
calls, workspaces and strides of every legal kind, values that are not finite, large caps, error
words with several bits, arguments that do not fit an int. Bounds as in test_paged.py."""
import ctypes
import math

import numpy as np
import pytest

from exact_io_aware_45_b200 import fa
from oracle import paged as orc
from test_paged import G, TYPES, U, build, check, fwd, ints, view


# ------------------------------------------------------------------ workspaces

def cache_of(dtype, d):
    return view(dtype=fa.FA_BF16 if dtype == "bf16" else fa.FA_F32, d=d, page_stride=2 * 16 * d)


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("T,shared", [(1, 0), (1, 32), (40, 0), (300, 64)])
def test_workspace_has_room_for_its_own_alignment(dtype, d, T, shared):
    """The partial results are whole multiples of 256 bytes and begin on a 32-byte boundary; a
    workspace is 16-byte aligned, so its size has 16 bytes more."""
    c = ctypes.byref(cache_of(dtype, d))
    size = fa.fa_paged_workspace_size(c, 2, T, 4, shared)
    assert size > 0 and size % 256 >= 16
    # a workspace that begins in the middle of 32 bytes and lacks the room is refused
    assert fwd(cache_of(dtype, d), shared or None, T=T, ws=G + 16,
               wsb=size - 16) == fa.FA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 128),
                                     ("f32", 16)])
@pytest.mark.parametrize("B,T,Hq,shared", [(3, 1, 4, 0), (3, 40, 4, 0), (2, 150, 2, 0), (9, 20, 4, 64),
                                           (5, 1, 4, 64), (40, 4, 8, 256)])
def test_workspaces_aligned_to_16_bytes(dtype, d, B, T, Hq, shared):
    """Partial results of every kernel in a workspace that no larger power of two divides, with
    nothing written outside of it."""
    import torch
    lens = [shared + 700 + 90 * b for b in range(B)]
    cache, seqs, dense = build(lens, 2, d, 16, dtype, shared=shared)
    q = torch.randn(B, Hq, T, d, device="cuda").to(cache.dtype)
    size = fa.fa_paged_workspace_size(cache._ref, B, T, Hq, shared)
    buf = torch.full((size + 1024,), 0xa5, dtype=torch.uint8, device="cuda")
    at = -buf.data_ptr() % 256 + 16
    kw = dict(workspace=buf[at:at + size])
    o, lse = (fa.forward_shared(q, cache, 0, shared, seqs, **kw) if shared else
              fa.forward_paged(q, cache, 0, seqs, **kw))
    cache.check()
    check(o, lse, q, dense, lens, 0, dtype, 1 / math.sqrt(d))
    assert (buf[:at] == 0xa5).all() and (buf[at + size:] == 0xa5).all()


# ------------------------------------------------------------------ empty calls

@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("B,T,shared", [(2, 0, 0), (2, 0, 16), (0, 1, 0), (0, 1, 16), (0, 40, 16),
                                        (0, 0, 0), (0, 0, 16)])
def test_empty_calls_have_a_workspace(dtype, d, B, T, shared):
    c = cache_of(dtype, d)
    assert fa.fa_paged_workspace_size(ctypes.byref(c), B, T, 4, shared) > 0
    assert fwd(c, shared or None, B=B, T=T, Q=0) == fa.FA_OK
    assert fa.fa_last_launch_count() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", TYPES)
def test_empty_calls_in_python(dtype, d):
    import torch
    cache, seqs, _ = build([20, 30], 2, d, 16, dtype)
    for B, T in ((0, 1), (2, 0), (0, 0), (0, 5)):
        q = torch.zeros(B, 4, T, d, dtype=cache.dtype, device="cuda")
        for o, lse in (fa.forward_paged(q, cache, 0, seqs[:B]),
                       fa.forward_shared(q, cache, 0, 16, seqs[:B])):
            assert o.shape == q.shape and lse.shape == (B, 4, T)
    none = seqs[:0]
    assert cache.extend(none, 3).numel() == 0
    cache.fork(none, none), cache.free(none), cache.copy_pages(none, none)
    new = torch.zeros(0, 2, d, dtype=cache.dtype, device="cuda")
    cache.write(0, new, new, none, none)
    cache.check()


# ------------------------------------------------------------------ values that are not finite

NAN_CASES = [("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 128), ("f32", 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", NAN_CASES)
@pytest.mark.parametrize("T,shared", [(1, 0), (3, 0), (40, 0), (160, 0), (1, 256), (4, 256)])
@pytest.mark.parametrize("cap", [0.0, 5.0, 1e4])
def test_nan_is_not_lost(dtype, d, T, shared, cap):
    """A NaN in a query row makes that row NaN and leaves the others as they are, to the bit (a
    row's arithmetic is its own); a NaN in a key makes every row NaN that sees it."""
    import torch
    B, Hq = (12, 8) if shared else (3, 4)
    lens = [shared + T + 200 + 60 * b for b in range(B)]
    cache, seqs, dense = build(lens, 2, d, 16, dtype, shared=shared)
    q = torch.randn(B, Hq, T, d, device="cuda").to(cache.dtype)

    def call():
        return (fa.forward_shared(q, cache, 0, shared, seqs, softcap=cap) if shared else
                fa.forward_paged(q, cache, 0, seqs, softcap=cap))

    o, lse = call()
    assert o.isfinite().all() and lse.isfinite().all()
    b, h, t = 1, Hq - 1, T // 2
    q[b, h, t, d // 3] = math.nan
    o2, lse2 = call()
    assert o2[b, h, t].isnan().all() and lse2[b, h, t].isnan()
    o2[b, h, t], lse2[b, h, t] = o[b, h, t], lse[b, h, t]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    q[b, h, t, d // 3] = 0
    o, lse = call()
    j = lens[b] - 1                                      # the last token of sequence b, KV head 1
    page = int(cache.table[int(seqs[b]), j // 16])
    cache.k[0, page, 1, j % 16, 3] = math.nan
    o2, lse2 = call()
    hit = (o2[b, Hq // 2:, T - 1], lse2[b, Hq // 2:, T - 1])
    assert all(x.isnan().all() for x in hit)
    o2[b, Hq // 2:, T - 1], lse2[b, Hq // 2:, T - 1] = (
        o[b, Hq // 2:, T - 1], lse[b, Hq // 2:, T - 1])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    cache.check()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,B,causal", [(200, 1, True), (640, 1, False), (1500, 8, True)])
def test_nan_query_of_the_dense_forward_under_a_cap(d, N, B, causal):
    """The row is NaN in O, and in LSE what it is without a cap."""
    import torch
    q, k, v = (torch.randn(B, 4, N, d, device="cuda").bfloat16() for _ in range(3))
    q[0, 1, 77, 5] = math.nan
    _, plain = fa.forward_mod(q, k, v, fa.mods(), causal=causal)
    o, lse = fa.forward_mod(q, k, v, fa.mods(softcap=3.0), causal=causal)
    assert o[0, 1, 77].isnan().all()
    assert torch.equal(lse[0, 1, 77].nan_to_num(9.0), plain[0, 1, 77].nan_to_num(9.0))
    o[0, 1, 77], lse[0, 1, 77] = 0, 0
    assert o.isfinite().all() and lse.isfinite().all()


# ------------------------------------------------------------------ what no query sees

def hide(cache, seqs, lens, shared, T, wl, value=math.nan):
    """Overwrites the shared rows that no query of the call sees."""
    page = cache.page_size
    reach = [min(n, shared) for n in lens]
    table = cache.table[int(seqs[reach.index(max(reach))])].tolist()
    seen = np.zeros(shared, dtype=bool)
    for n in lens:
        if n:
            seen[max(0, n - T - wl):min(n, shared)] = True
    for j in np.flatnonzero(~seen):
        if table[j // page] >= 0:
            cache.k[:, table[j // page], :, j % page] = value
            cache.v[:, table[j // page], :, j % page] = value
    return int((~seen).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 16), ("f32", 128),
                                     ("f32", 64), ("f32", 16)])
@pytest.mark.parametrize("lens,Hq,T", [
    ([1024], 2, 1), ([1030, 0], 4, 1), ([0, 1030, 1100, 0], 8, 3),      # padding
    ([1040, 100], 4, 1), ([100, 417, 1040, 0], 8, 2),                   # holes between windows
    ([7, 0, 300, 555, 1024, 1025, 1200] * 5, 8, 2),
    ([90, 400, 0], 4, 2), ([500, 130, 131] * 20, 8, 3)])                # none behind the prefix
@pytest.mark.parametrize("wl,cap", [(0, 0.0), (37, 0.0), (200, 9.0)])
def test_shared_rows_that_no_query_sees(dtype, d, lens, Hq, T, wl, cap):
    """Padding and short sequences behind a prefix under a window: the rows that no query sees hold
    NaN, before the windows and between them."""
    import torch
    shared = 1024
    cache, seqs, dense = build(lens, 2, d, 32, dtype, shared=shared)
    assert hide(cache, seqs, lens, shared, T, wl) > 0
    q = torch.randn(len(lens), Hq, T, d, device="cuda").to(cache.dtype)
    o, lse = fa.forward_shared(q, cache, 0, shared, seqs, window_left=wl, softcap=cap)
    cache.check()
    check(o, lse, q, dense, lens, 0, dtype, 1 / math.sqrt(d), wl=wl, cap=cap)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,reps", [("bf16", 128, 1), ("bf16", 64, 9), ("f32", 64, 1),
                                          ("f32", 32, 9)])
def test_shared_window_with_padding_out_of_range(dtype, d, reps):
    import torch
    lens = [300, 512, 700] * reps
    cache, seqs, dense = build(lens, 2, d, 32, dtype, shared=256)
    assert hide(cache, seqs, lens, 256, 1, 40) > 0
    slots = torch.cat([ints([-1]), seqs, ints([10 ** 6])])
    q = torch.randn(len(slots), 8, 1, d, device="cuda").to(cache.dtype)
    o, lse = fa.forward_shared(q, cache, 0, 256, slots, window_left=40)
    cache.check()
    check(o[1:-1], lse[1:-1], q[1:-1], dense, lens, 0, dtype, d ** -0.5, wl=40)
    assert not o[[0, -1]].any() and torch.isneginf(lse[[0, -1]]).all()


# ------------------------------------------------------------------ large caps

def check_cap(o, lse, q, dense, lens, dtype, scale, cap):
    """As check, but the cap costs a score at most 2^-19 of its own size: tanh off by 1.5e-6 of its
    value, products by three roundings."""
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    T, d = o.shape[2:]
    for b, n in enumerate(lens):
        k, v = (x[0].float().cpu().numpy() for x in dense[b])
        O, L, A, X = orc.attend(q[b].float().cpu().numpy(), k, v, T, n - T, scale, softcap=cap)
        dx = (2 * (d + 8) * U + 2.0 ** -19) * X
        tol = A * (2 * dx + 2 * (n + 64) * U + 2.0 ** -20)[..., None]
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * (A + np.abs(O))
        off = (np.abs(o[b] - O) - tol).max()
        assert off <= 0, f"sequence {b}: O off by {off:.3e} too much"
        off = (np.abs(lse[b] - L) - dx - (n + 64) * U - 2.0 ** -20 * (1 + np.abs(L))).max()
        assert off <= 0, f"sequence {b}: LSE off by {off:.3e} too much"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("B,T,shared", [(3, 1, 0), (3, 5, 0), (3, 40, 0), (2, 150, 0), (20, 4, 256)])
@pytest.mark.parametrize("cap", [0.05, 1e3, 1e6, 3e38])
@pytest.mark.parametrize("scale", [None, -1e-3])
def test_caps_of_every_size(dtype, d, B, T, shared, cap, scale):
    """A cap far above the scores changes them by less than their rounding."""
    import torch
    lens = [shared + T + 80 + 37 * b for b in range(B)]
    cache, seqs, dense = build(lens, 2, d, 16, dtype, shared=shared)
    scale = 1 / math.sqrt(d) if scale is None else scale
    q = torch.randn(B, 8, T, d, device="cuda").to(cache.dtype)
    kw = dict(scale=scale, softcap=cap)
    o, lse = (fa.forward_shared(q, cache, 0, shared, seqs, **kw) if shared else
              fa.forward_paged(q, cache, 0, seqs, **kw))
    cache.check()
    check_cap(o, lse, q, dense, lens, dtype, scale, cap)


# ------------------------------------------------------------------ one workspace, many calls

@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("T,shared", [(1, 0), (40, 0), (1, 512), (6, 512)])
def test_calls_that_follow_on_one_workspace(dtype, d, T, shared):
    """Two queries in turn on one workspace, back to back and captured: each result is its own,
    none is joined from what the call before left there."""
    import torch
    lens = [shared + 900 + 50 * b for b in range(7)]
    cache, seqs, dense = build(lens, 2, d, 16, dtype, shared=shared)
    qs = [torch.randn(7, 8, T, d, device="cuda").to(cache.dtype) for _ in range(2)]
    ws = torch.empty(fa.fa_paged_workspace_size(cache._ref, 7, T, 8, shared), dtype=torch.uint8,
                     device="cuda")

    def call(q, **kw):
        return (fa.forward_shared(q, cache, 0, shared, seqs, **kw) if shared else
                fa.forward_paged(q, cache, 0, seqs, **kw))

    want = [call(q) for q in qs]
    for q, w in zip(qs, want):
        check(*w, q, dense, lens, 0, dtype, 1 / math.sqrt(d))
    n = 60
    got = [[torch.empty_like(x) for x in want[0]] for _ in range(n)]

    def run():
        for i, (o, lse) in enumerate(got):
            call(qs[i % 2], out=o, lse=lse, workspace=ws)

    run()
    first = [[x.clone() for x in g] for g in got]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for i in range(n):
        for x, y, w in zip(first[i], got[i], want[i % 2]):
            assert torch.equal(x, w) and torch.equal(y, w)


# ------------------------------------------------------------------ error words

@pytest.mark.gpu
def test_a_refusal_and_a_timeout_are_both_reported():
    """A refused extension and a wait that ran out between two checks: neither hides the other."""
    import torch
    lens = [400, 401, 402]
    cache, seqs, dense = build(lens, 2, 64, 16, "bf16")
    q = torch.randn(3, 8, 30, 64, device="cuda").bfloat16()
    fa.forward_paged(q, cache, 0, seqs)
    torch.cuda.synchronize()
    assert (cache.extend(ints([0, 0]), 1) == -1).all()
    assert fa.fa_debug_set_stall(fa.FA_STALL_FWD, 4_000_000) == fa.FA_OK
    try:
        fa.forward_paged(q, cache, 0, seqs)
        torch.cuda.synchronize()
    finally:
        fa.fa_debug_set_stall(0, 0)
    found = []
    for _ in range(2):
        with pytest.raises(fa.FaError) as e:
            cache.check()
        found.append(e.value.status)
    assert sorted(found) == [fa.FA_ERR_TIMEOUT, fa.FA_ERR_CACHE]
    cache.check()
    assert not cache.err.any()
    o, lse = fa.forward_paged(q, cache, 0, seqs)
    check(o, lse, q, dense, lens, 0, "bf16", 0.125)


@pytest.mark.gpu
@pytest.mark.parametrize("word,want", [(1, [fa.FA_ERR_TIMEOUT]), (2, [fa.FA_ERR_CUDA]),
                                       (4, [fa.FA_ERR_CACHE]), (3, [fa.FA_ERR_TIMEOUT]),
                                       (7, [fa.FA_ERR_TIMEOUT, fa.FA_ERR_CACHE])])
def test_error_words(word, want):
    """Each status once, and the word is clear afterwards."""
    import torch
    err = torch.zeros(64, dtype=torch.int32, device="cuda")
    err[0] = word
    for w in want + [fa.FA_OK]:
        assert fa.fa_get_device_error(err.data_ptr(), torch.cuda.current_stream().cuda_stream) == w
    assert not err.any()


# ------------------------------------------------------------------ strides of single entries

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_of_dimensions_of_one_entry_do_not_matter(dtype):
    """One KV head kept as [pages, page, 1, d], one layer, one page: the same bytes, other strides."""
    import torch
    lens = [70, 5]
    cache, seqs, dense = build(lens, 1, 64, 16, dtype)
    q = torch.randn(2, 4, 1, 64, device="cuda").to(cache.dtype)
    want = fa.forward_paged(q, cache, 0, seqs)
    rest = (cache.table, cache.lens, cache.refs)
    P = cache.pages
    views = [cache.k[0, :, 0].unsqueeze(2).transpose(1, 2)[None],              # [1, P, 1, 16, 64]
             cache.k.as_strided((1, P, 1, 16, 64), (3, 1024, 7, 64, 1))]
    for k in views:
        for v in (cache.v, cache.v.as_strided(k.shape, (5, 1024, 1, 64, 1))):
            o, lse = fa.forward_paged(q, fa.PagedCache(k, v, *rest), 0, seqs)
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    small = fa.PagedCache.new(1, 1, 1, 16, 64, 1, 1, cache.dtype)
    k, v = (x.as_strided((1, 1, 1, 16, 64), (1, 1, 1, 64, 1)) for x in (small.k, small.v))
    one = fa.PagedCache(k, v, small.table, small.lens, small.refs)
    pos = one.extend(ints([0]), 9)
    new = torch.randn(9, 1, 64, device="cuda").to(cache.dtype)
    one.write(0, new, new, ints([0]), pos)
    one.check()
    assert torch.equal(small.k[0, 0, 0, :9], new[:, 0])
    for stride in ((0, 1024, 0, 64, 2), (0, 1025, 0, 64, 1), (0, 1024, 0, 0, 1)):
        bad = cache.k.as_strided((1, P - 1, 1, 16, 64), stride)
        with pytest.raises(ValueError):
            fa.PagedCache(bad, bad, cache.table, cache.lens, cache.refs[:-1])


# ------------------------------------------------------------------ numbers that do not fit an int

@pytest.mark.gpu
@pytest.mark.parametrize("n", [1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 31) - 1, 1 << 63, 1 << 70])
def test_numbers_that_do_not_fit_are_refused(n):
    """None is taken modulo 2^32."""
    import torch
    cache, seqs, _ = build([20, 30], 2, 64, 16, "bf16")
    q = torch.randn(2, 4, 1, 64, device="cuda").bfloat16()
    new = torch.zeros(2, 2, 64, device="cuda").bfloat16()
    keep = cache.lens.clone()
    for call in (lambda: cache.extend(seqs, n), lambda: fa.forward_paged(q, cache, n, seqs),
                 lambda: fa.forward_paged(q, cache, 0, seqs, window_left=n),
                 lambda: fa.forward_shared(q, cache, 0, n, seqs),
                 lambda: fa.forward_shared(q, cache, n, 16, seqs),
                 lambda: cache.write(n, new, new, seqs, keep[:2])):
        with pytest.raises((ValueError, fa.FaError)):
            call()
    assert torch.equal(cache.lens, keep)
    cache.check()


# ------------------------------------------------------------------ the longest lists

def test_more_slots_than_loops_can_count():
    """Loops over slots step past their number, in 32 bits."""
    for seqs in ((1 << 31) - 1, (1 << 31) - 4096):
        c = ctypes.byref(view(seqs=seqs, seq_pages=1))
        assert fa.fa_cache_workspace_size(c, 1) == 0
        assert fa.fa_cache_free(c, G, 1, G, 1 << 40, 0) == fa.FA_ERR_UNSUPPORTED
        assert fa.fa_paged_workspace_size(c, 1, 1, 4, 0) == 0


@pytest.mark.gpu
def test_write_of_almost_2_31_rows():
    """The rows of a skipped sequence, up to the largest count, and one that is written."""
    import torch
    total = (1 << 31) - 1
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB free")
    cache = fa.PagedCache.new(1, 4, 1, 16, 16, 2, 2)
    pos = cache.extend(ints([0]), 3)
    new = torch.empty(total, 1, 16, dtype=torch.bfloat16, device="cuda")
    new[-3:] = torch.arange(3, device="cuda").bfloat16()[:, None, None] + 1
    cache.write(0, new, new, ints([1, 0]), torch.cat([ints([-1]), pos]),
                ints([0, total - 3, total]))
    cache.check()
    assert cache.k[0, 0, 0, :4, 0].tolist() == [1, 2, 3, 0] and not cache.k[0, 1:].any()


def test_empty_calls_of_many_heads():
    """Sizes whose products pass 32 bits where a factor is 0."""
    heads = 1 << 20
    c = ctypes.byref(view(Hkv=heads, d=16, page_stride=heads * 16 * 16))
    for B, T in ((65535, 0), (0, 1 << 18)):
        assert 0 < fa.fa_paged_workspace_size(c, B, T, heads, 0) < 1 << 20
