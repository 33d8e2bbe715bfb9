"""sv_prefix_attention against sv_window_attention's definition in 64 bits, its refusals (CPU) and data errors."""
import ctypes
import math

import pytest
import torch

from speculative_decoding_verification_27_gb300 import api, build
from test_attention import BF, F32, INF, Case
from test_attention8 import E8, Case8, late_candidates
from test_cache import FAKE, ODD, _cache, _seqs


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return api.load()


def _call(lib, **kw):
    a = dict(q=FAKE, qs=256, heads=4, R=10, cache=_cache(), layer=0, seqs=_seqs(), n_groups=1, cg=FAKE, pl=FAKE, n_cand=3, cu=FAKE, cand=None,
             scale=0.1, out=FAKE, os=256, lse=None, ws=FAKE, wsb=1 << 30, status=None)
    a.update(kw)
    return lib.sv_prefix_attention(*a.values(), None)


def test_host_validation(lib):
    E, OK = api.SV_ERR_INVALID_ARG, api.SV_OK
    assert _call(lib, R=0) == OK and _call(lib, seqs=_seqs(n=0), n_cand=0) == OK and _call(lib, R=0, n_groups=0, cg=None, pl=None) == OK
    for bad in (dict(n_groups=-1), dict(cg=None), dict(pl=None), dict(cg=ODD), dict(pl=ODD), dict(q=None), dict(qs=255), dict(heads=3), dict(R=-1),
                dict(layer=2), dict(n_cand=2), dict(cu=None, cand=FAKE), dict(scale=math.nan), dict(out=None), dict(os=64), dict(lse=ODD),
                dict(ws=None), dict(ws=FAKE + 8), dict(wsb=0), dict(status=ODD), dict(cache=_cache(head_dim=32, head_stride=32))):
        assert _call(lib, **bad) == E, bad
    size = lib.sv_prefix_attention_workspace_size
    least = size(_cache(), 4, 10, 3, 1)
    assert _call(lib, wsb=least - 1) == E
    assert least >= lib.sv_window_attention_workspace_size(_cache(), 4, 10) + 10 * 4 * 66 * 4
    for bad in ((0, 10, 3, 1), (4, -1, 3, 1), (4, 10, -1, 1), (4, 10, 3, -1)):
        assert size(_cache(), *bad) == 0
    assert size(_cache(head_dim=32, head_stride=32), 4, 10, 3, 1) == 0


# ---------------------------------------------------------------------------
def share(c, groups):
    """Lets the sequences s0 .. s1-1 of a case begin with the same p tokens, for (s0, s1, p) of groups: whole pages are the first
    sequence's, a part of one is copied; the pages that they had instead hold NaN."""
    pools = [*c.raw, *c.scale] if isinstance(c, Case8) else [c.k, c.v]
    for s0, s1, p in groups:
        for b in range(s0 + 1, s1):
            for i in range(p // c.page):
                for x in pools:
                    x[0, c.table[b, i]] = 0x7F if x.dtype == torch.uint8 else math.nan
                c.table[b, i] = c.table[s0, i]
            if p % c.page:
                for x in pools:
                    x[0, c.table[b, p // c.page], : p % c.page] = x[0, c.table[s0, p // c.page], : p % c.page]
    if isinstance(c, Case8):
        c.dequantise()
    c.groups = groups
    return c


def prefix_args(c):
    edge = [c.groups[0][0]] if c.groups else [0]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for s0, s1, _ in c.groups:
        assert s0 == edge[-1]
        edge.append(s1)
    return (*c.args[:5], i32(edge), i32([p for _, _, p in c.groups]), *c.args[5:])


def check(c, **kw):
    Case.run(c, **kw) if not isinstance(c, Case8) else Case8.run(c, **kw)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((c.R, c.Hq, c.D), 7.0, dtype=c.dtype, device="cuda")
    lse = torch.full((c.R, c.Hq), 7.0, device="cuda")
    api.sv_prefix_attention(*prefix_args(c), out=out, out_lse=lse, status=status, **kw)
    assert int(status) == 0
    want, want_l, tol, tol_l = c.reference(kw.get("scale"))
    out, lse = out.cpu().double(), lse.cpu().double()
    assert bool(((out - want).abs() <= tol).all()), float(((out - want).abs() - tol).max())
    assert bool(((lse - want_l).abs() <= tol_l).all()), float(((lse - want_l).abs() - tol_l).max())


def make(dtype, ctx, lens, Hq, Hkv, D, page, groups, **kw):
    c = Case8(ctx, lens, Hq, Hkv, D, page, **kw) if dtype == E8 else Case(ctx, lens, Hq, Hkv, D, page, dtype, **kw)
    return share(c, groups)


TYPES = [BF, F32, E8]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (8, 2, 128), (6, 2, 64), (64, 1, 64), (4, 4, 128), (32, 1, 128), (10, 2, 64)])
@pytest.mark.parametrize("page", [1, 7, 64])
def test_groups(cuda_lib, dtype, Hq, Hkv, D, page):
    """Prefixes around the tiles' and pages' edges, groups of one, without a prefix, with an empty window, and sequences of no group."""
    ctx = [40, 63, 70, 64, 90, 5, 130, 129, 131, 200, 7, 1, 0, 12]
    lens = [[1], [3], [2], [1], [4], [2], [1, 2], [5], [], [1], [1], [2], [1], [1]]
    groups = [(1, 3, 63), (3, 5, 64), (5, 6, 5), (6, 9, 129), (9, 11, 0), (11, 11, 3), (11, 12, 1)]
    check(make(dtype, ctx, lens, Hq, Hkv, D, page, groups, seed=Hq * 10 + page))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 64, 16), (4, 1, 128, 5), (16, 2, 128, 16), (64, 2, 64, 16)])
def test_long_prefixes(cuda_lib, dtype, Hq, Hkv, D, page):
    """Prefixes that are split over the machine, windows of candidates, a sequence that has nothing but the prefix."""
    ctx = [2500, 2600, 2501, 2500, 300, 777, 800, 800]
    lens = [[2], [1, 3], [4], [1], [2], [1], [2, 2, 2], [1]]
    c = make(dtype, ctx, lens, Hq, Hkv, D, page, [(0, 4, 2500), (4, 5, 100), (5, 8, 770)], seed=D)
    check(c)
    args = prefix_args(c)
    want = api.sv_prefix_attention(*args, want_lse=True)
    for _ in range(3):
        got = api.sv_prefix_attention(*args, want_lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # Without groups the call is sv_window_attention.
    empty = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = api.sv_prefix_attention(*args[:5], empty, empty[:0], *args[7:], want_lse=True)
    b = api.sv_window_attention(*c.args, want_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows(cuda_lib, dtype, D):
    """A group of many sequences, so that its rows fill several row tiles, beside one of a few."""
    gen = torch.Generator().manual_seed(D)
    n = 60
    ctx = [300 + int(x) for x in torch.randint(0, 70, (n,), generator=gen)]
    lens = [[int(x)] for x in torch.randint(1, 9, (n,), generator=gen)]
    check(make(dtype, ctx, lens, 8, 2, D, 16, [(0, 50, 300), (50, 57, 290)], seed=D, cands=False))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq", [4, 64])
@pytest.mark.parametrize("scale,heavy", [(None, True), (0.0, False), (-0.2, False), (2.0, False)])
def test_peaked_rows_and_scales(cuda_lib, dtype, Hq, scale, heavy):
    """The largest scores in the prefix and behind it, a scale of zero, a negative one."""
    c = make(dtype, [300, 340, 310], [[3], [2], [4]], Hq, 2, 64, 16, [(0, 3, 300)], seed=7, heavy=heavy)
    pool = c.scale[0] if dtype == E8 else c.k
    first = c.table[0].long()
    pool[0, first[10]] *= 4.0          # tokens of the prefix
    pool[0, int(c.table[1, 20])] *= 6.0  # of the second sequence's own
    if dtype == E8:
        c.dequantise()
    check(c, **({} if scale is None else {"scale": scale}))


@pytest.mark.gpu
@pytest.mark.parametrize("low", [False, True])
@pytest.mark.parametrize("Hq,D", [(2, 64), (4, 128)])
def test_rows_that_see_nothing_of_the_first_tiles(cuda_lib, Hq, D, low):
    """Behind the prefix, rows whose own tokens begin a tile or more into their windows."""
    check(share(late_candidates(Hq, D, low, prefix=200), [(0, 40, 200)]), **({"scale": 0.5} if low else {}))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,last", [(8, [[3], [1]]), (24, [[1]]), (4, [[5, 4], [2]])])
def test_last_windows_of_few_rows(cuda_lib, dtype, D, Hq, last):
    """Windows that leave half of a row tile empty, the batch's last ones, with no row behind them and a workspace of just the size
    that is asked for: the half without a row has nothing in it."""
    rows = 64 // Hq
    c = make(dtype, [150, 140, 201, 170, 141, 139, 144][: 5 + len(last)], [[rows + b % 2] for b in range(5)] + last, Hq, 1, D, 16,
             [(0, 5 + len(last), 139)], seed=D + Hq, spare=0)
    c.run()
    nbytes = api.load().sv_prefix_attention_workspace_size(c.args[1]._ref, Hq, c.R, len(c.ctx), 1)
    check(c, workspace=torch.empty(nbytes, dtype=torch.uint8, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("low", [False, True])
@pytest.mark.parametrize("Hq,D", [(8, 64), (8, 128)])
def test_rows_that_see_nothing_in_two_halves(cuda_lib, Hq, D, low):
    """Row tiles of 64, whose halves move their references by themselves."""
    check(share(late_candidates(Hq, D, low, prefix=200), [(0, 40, 200)]), **({"scale": 0.5} if low else {}))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout,q_pad", [("hnd", 0), ("both", 64)])
def test_layouts_and_strides(cuda_lib, dtype, layout, q_pad):
    check(make(dtype, [140, 203, 150, 141], [[4], [2, 3], [1], [6]], 8, 4, 64, 16, [(0, 2, 140), (2, 4, 141)], seed=3, layout=layout, q_pad=q_pad))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_single_tokens_and_thousands_of_sequences(cuda_lib, dtype):
    """cu_draft of None; more sequences and groups than a CTA has threads."""
    n = 2200
    c = make(dtype, [20 + b % 5 for b in range(n)], [[1]] * n, 2, 1, 64, 16, [(b, b + 2, 20 - b % 4) for b in range(0, n, 2)], seed=3, cands=False)
    check(c)
    args = prefix_args(c)
    a = api.sv_prefix_attention(*args, want_lse=True)
    b = api.sv_prefix_attention(*args[:7], want_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_data_errors(cuda_lib, dtype):
    """Groups that cannot be shared are attended to sequence by sequence; windows that cannot be served are left alone, with their
    group's others served; hidden pages of a prefix hide it from all."""
    c = make(dtype, [100, 120, 90, 95], [[2], [3], [1], [2]], 4, 2, 64, 8, [(0, 2, 100), (2, 4, 90)], seed=12, cands=False)
    check(c)
    q, cache, layer, table, ctx, cg, pl, cu, cand = prefix_args(c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    alone = api.sv_window_attention(*c.args, want_lse=True)
    for edges in ([0, 3, 2], [-1, 2, 4], [0, 2, 5], [0, 1 << 30, 4]):
        status.zero_()
        got = api.sv_prefix_attention(q, cache, layer, table, ctx, i32(edges), pl, cu, cand, want_lse=True, status=status)
        assert int(status) == api.SV_DATA_BAD_OFFSETS
        assert torch.equal(got[0], alone[0]) and torch.equal(got[1], alone[1])
    for lengths in ([101, 90], [-1, 90], [1 << 30, 90]):
        status.zero_()
        got = api.sv_prefix_attention(q, cache, layer, table, ctx, cg, i32(lengths), cu, cand, want_lse=True, status=status)
        assert int(status) == api.SV_DATA_BAD_SEQ
        assert torch.equal(got[0][:5], alone[0][:5]) and (got[1][5:8] - alone[1][5:8]).abs().max() < 1e-4
    # A sequence of the first group with a bad length, then a window that does not fit its table.
    for bad, bits in ((-1, api.SV_DATA_BAD_SEQ), (table.shape[1] * 8 - 1, api.SV_DATA_BAD_SEQ | api.SV_DATA_BAD_PAGE)):
        status.zero_()
        x = ctx.clone()
        x[1] = bad
        out = torch.full_like(q, 7.0)
        api.sv_prefix_attention(q, cache, layer, table, x, cg, pl, cu, cand, out=out, status=status)
        assert int(status) == bits
        assert torch.equal(out[:2], alone[0][:2]) and bool((out[2:5] == 7).all()) and (out[5:8].float() - alone[0][5:8].float()).abs().max() < 0.05
    # The prefix's pages out of range: its sequences see their own tokens only.
    status.zero_()
    broken = table.clone()
    broken[0, :] = 1 << 20
    got = api.sv_prefix_attention(q, cache, layer, broken, ctx, cg, pl, cu, cand, want_lse=True, status=status)
    assert int(status) == api.SV_DATA_BAD_PAGE
    assert bool((got[0][:2] == 0).all()) and bool((got[1][:2] == -INF).all())
    keep = torch.arange(100, 121)
    k = c.k[0][c.table[1].long()[keep // 8], keep % 8].double().repeat_interleave(2, 1)
    s = torch.einsum("hd,thd->ht", c.q[2].double(), k) / 8
    assert (torch.logsumexp(s, 1) - got[1][2].cpu().double()).abs().max() < 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_graphs_and_streams(cuda_lib, dtype):
    """Captured calls replay together, on new lengths and prefixes; calls on streams of the caller's give the same bits."""
    c = make(dtype, [900, 930, 950, 40], [[2], [4], [1], [3]], 8, 2, 64, 16, [(0, 3, 896)], seed=13)
    check(c)
    args = prefix_args(c)
    want = api.sv_prefix_attention(*args, want_lse=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [api.sv_prefix_attention(*args, want_lse=True, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)
    graphs, sets = [], []
    for _ in range(2):
        mine = [x.clone() if i in (4, 6) else x for i, x in enumerate(args)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = api.sv_prefix_attention(*mine, want_lse=True)
        graphs.append((g, o))
        sets.append(mine)
    sets[1][4].copy_(torch.tensor([800, 810, 805, 30], dtype=torch.int32))
    sets[1][6].copy_(torch.tensor([777], dtype=torch.int32))
    short = api.sv_prefix_attention(*sets[1], want_lse=True)
    torch.cuda.synchronize()
    for (g, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1][0], want[0]) and torch.equal(graphs[1][1][0], short[0])
    assert torch.equal(graphs[0][1][1], want[1]) and torch.equal(graphs[1][1][1], short[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_forks_of_a_prompt(cuda_lib, dtype):
    """A prompt appended once, forked, and a step of its forks: reserve copies the partly filled page, rope and append write the forks'
    rows, and the attention with the shared prefix is that of each fork by itself."""
    torch.manual_seed(1)
    row, H, D, page, n, p = (F32 if dtype == F32 else BF), 2, 64, 16, 6, 203
    k = torch.zeros(1, 60, page, H, D, device="cuda").to(dtype)
    cache = api.KVCache(k, k.clone())
    table = torch.full((n + 1, 16), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    angle = torch.arange(300, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    kw = dict(cos_sin=torch.cat([angle.cos(), angle.sin()], 1), status=status)

    def rows(R, heads):
        return torch.randn(R, heads, D, device="cuda").to(row)

    api.sv_cache_reserve(cache, table[:1], ctx[:1], torch.tensor([0, p - 1], dtype=torch.int32, device="cuda"), status=status)
    api.sv_rope_append(rows(p, 4), rows(p, H), rows(p, H), cache, 0, table[:1], ctx[:1], torch.tensor([0, p - 1], dtype=torch.int32, device="cuda"), **kw)
    api.sv_cache_commit(cache, table[:1], ctx[:1], torch.tensor([0, p - 1], dtype=torch.int32, device="cuda"),
                        torch.tensor([p], dtype=torch.int32, device="cuda"), status=status)
    api.sv_cache_fork(cache, table, ctx, torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(1, n + 1, dtype=torch.int32, device="cuda"),
                      status=status)
    table, ctx = table[1:], ctx[1:]
    cu = torch.arange(0, 3 * n + 1, 3, dtype=torch.int32, device="cuda")
    R = 4 * n
    for step in range(2):
        api.sv_cache_reserve(cache, table, ctx, cu, status=status)
        q = api.sv_rope_append(rows(R, 4), rows(R, H), rows(R, H), cache, 0, table, ctx, cu, **kw)
        group = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        got = api.sv_prefix_attention(q, cache, 0, table, ctx, group, torch.tensor([p], dtype=torch.int32, device="cuda"), cu, want_lse=True, status=status)
        want = api.sv_window_attention(q, cache, 0, table, ctx, cu, want_lse=True, status=status)
        assert int(status) == 0
        assert (got[1] - want[1]).abs().max() < 1e-4 and (got[0].float() - want[0].float()).abs().max() < (1e-4 if dtype == F32 else 0.03)
        api.sv_cache_commit(cache, table, ctx, cu, torch.randint(1, 5, (n,), dtype=torch.int32, device="cuda"), status=status)


@pytest.mark.gpu
def test_binding_refuses(cuda_lib):
    c = make(BF, [30, 31], [[2], [1]], 4, 2, 64, 8, [(0, 2, 30)], seed=4, cands=False)
    c.run()
    args = list(prefix_args(c))
    for i, bad in ((0, args[0].float()), (0, args[0][:, :, :32]), (5, args[5].long()), (5, args[5][:1]), (6, args[6].float()), (6, args[6].cpu())):
        with pytest.raises(ValueError):
            api.sv_prefix_attention(*args[:i], bad, *args[i + 1:])
