"""sv_window_attention against its definition in 64 bits, its refusals (CPU),
its data errors, and a step of the cache, the attention, the verify call and
the log probabilities together."""
import ctypes
import math

import pytest
import torch

from speculative_decoding_verification_27_gb300 import api, build
from test_cache import FAKE, ODD, _cache, _seqs

INF = math.inf


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return api.load()


def _call(lib, **kw):
    a = dict(q=FAKE, qs=256, heads=4, R=10, cache=_cache(), layer=0, seqs=_seqs(), n_cand=3, cu=FAKE, cand=None, scale=0.1,
             out=FAKE, os=256, lse=None, ws=FAKE, wsb=1 << 30, status=None)
    a.update(kw)
    return lib.sv_window_attention(*a.values(), None)


def test_host_validation(lib):
    E, OK = api.SV_ERR_INVALID_ARG, api.SV_OK
    assert _call(lib, R=0) == OK and _call(lib, seqs=_seqs(n=0), n_cand=0) == OK
    for bad in (dict(q=None), dict(q=FAKE + 8), dict(qs=255), dict(qs=260), dict(qs=128), dict(heads=0), dict(heads=3),
                dict(heads=260, qs=1 << 20, os=1 << 20), dict(R=-1), dict(layer=-1), dict(layer=2), dict(n_cand=2), dict(cand=ODD),
                dict(cu=None, cand=FAKE), dict(cu=ODD), dict(scale=math.nan), dict(scale=INF), dict(out=None), dict(out=FAKE + 8),
                dict(os=260), dict(os=64), dict(lse=ODD), dict(ws=None), dict(ws=FAKE + 8), dict(wsb=0), dict(status=ODD),
                dict(cache=_cache(k=0)), dict(cache=_cache(head_dim=32, head_stride=32)), dict(cache=_cache(head_dim=256, head_stride=256)),
                dict(seqs=_seqs(table=0))):
        assert _call(lib, **bad) == E, bad
    assert lib.sv_window_attention_workspace_size(_cache(), 4, 10) >= 16
    assert lib.sv_window_attention_workspace_size(_cache(), 0, 10) == 0
    assert lib.sv_window_attention_workspace_size(_cache(), 4, -1) == 0


def test_scale_that_leaves_fp32_in_base_two(lib):
    """The scores are taken to base two: a scale has to stay finite times log2(e)."""
    assert _call(lib, scale=2.0 ** 127) == _call(lib, scale=-3e38) == api.SV_ERR_INVALID_ARG
    assert _call(lib, scale=2.0 ** 127, R=0) == api.SV_ERR_INVALID_ARG and _call(lib, scale=1.7e38, R=0) == api.SV_OK


# ---------------------------------------------------------------------------
# Against 64 bits
# ---------------------------------------------------------------------------
class Case:
    """Sequences of given lengths and windows over a shuffled pool: lens[b] is the list of request b's candidates' rows."""

    def __init__(self, ctx, lens, Hq, Hkv, D, page, dtype, seed=0, layout="nhd", spare=3, cands=True, heavy=False, q_pad=0):
        gen = torch.Generator().manual_seed(seed)
        self.ctx, self.lens, self.Hq, self.Hkv, self.D, self.page, self.dtype = ctx, lens, Hq, Hkv, D, page, dtype
        n = len(ctx)
        held = [-(-(c + sum(x)) // page) for c, x in zip(ctx, lens)]
        P = sum(held) + spare
        perm = torch.randperm(P, generator=gen).tolist()
        width = max(held + [1]) + 1
        table = [[-1] * width for _ in range(n)]
        for b, h in enumerate(held):
            for i in range(h):
                table[b][i] = perm.pop()
        self.table = torch.tensor(table, dtype=torch.int32)
        shape = (1, P, page, Hkv, D)
        nan = torch.full(shape, float("nan"))  # everything that no sequence holds
        k, v = nan.clone(), nan.clone()
        for b, h in enumerate(held):
            for t in range(ctx[b] + sum(lens[b])):
                p, i = table[b][t // page], t % page
                k[0, p, i] = torch.randn(Hkv, D, generator=gen)
                v[0, p, i] = torch.randn(Hkv, D, generator=gen)
        self.k, self.v = k.to(dtype), v.to(dtype)
        flat = [x for y in lens for x in y]
        self.R = sum(flat) + spare
        self.q = (torch.randn(self.R, Hq, D, generator=gen) * (6.0 if heavy else 1.5)).to(dtype)
        cu, cand = [0], [0]
        for y in lens:
            cand.append(cand[-1] + len(y))
            for x in y:
                cu.append(cu[-1] + x - 1)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.cand = torch.tensor(cand, dtype=torch.int32) if cands else None
        self.layout, self.q_pad = layout, q_pad

    def run(self, **kw):
        k, v = self.k.cuda(), self.v.cuda()
        if self.layout == "hnd":
            k, v = (x.transpose(2, 3).contiguous().transpose(2, 3) for x in (k, v))
        elif self.layout == "both":
            both = torch.stack([k, v], 2)
            k, v = both[:, :, 0], both[:, :, 1]
        cache = api.KVCache(k, v)
        q = self.q.cuda()
        if self.q_pad:
            wide = torch.zeros(self.R, self.Hq * self.D + self.q_pad, dtype=self.dtype, device="cuda")
            view = wide[:, : self.Hq * self.D].view(self.R, self.Hq, self.D)
            view.copy_(q)
            q = view
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((self.R, self.Hq, self.D), 7.0, dtype=self.dtype, device="cuda")
        lse = torch.full((self.R, self.Hq), 7.0, device="cuda")
        args = (q, cache, 0, self.table.cuda(), torch.tensor(self.ctx, dtype=torch.int32, device="cuda"), self.cu.cuda(),
                None if self.cand is None else self.cand.cuda())
        api.sv_window_attention(*args, out=out, out_lse=lse, status=status, **kw)
        assert int(status) == 0
        self.args = args
        return out.cpu(), lse.cpu()

    def reference(self, scale=None):
        """(out, lse, tolerance of out, of lse) in 64 bits.

        A score is a sum of D products in fp32 (tensor core sums are no worse
        than one rounding a product) with the rounding of the scale and of the
        exponent: d = (D + 8) 2^-24 scale sum|q k| relative to e^s; the running
        sums add n terms with one rescaling a term at most, each with the
        2^-22 of the exponential: (n + 64) 2^-22. With bf16 each weight is
        rounded to bf16 (2^-8) and so is the output."""
        scale = self.D ** -0.5 if scale is None else scale
        out = torch.full((self.R, self.Hq, self.D), 7.0, dtype=torch.float64)
        lse = torch.full((self.R, self.Hq), 7.0, dtype=torch.float64)
        tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
        g = self.Hq // self.Hkv
        r0 = 0
        for b, y in enumerate(self.lens):
            n = self.ctx[b] + sum(y)
            at = torch.arange(n)
            p = self.table[b].long()[at // self.page]
            k = self.k[0][p, at % self.page].double().repeat_interleave(g, 1)
            v = self.v[0][p, at % self.page].double().repeat_interleave(g, 1)
            begin = 0
            for x in y:
                for i in range(x):
                    seen = torch.cat([torch.arange(self.ctx[b]), self.ctx[b] + begin + torch.arange(i + 1)])
                    q = self.q[r0].double()
                    s = torch.einsum("hd,thd->ht", q, k[seen]) * scale
                    d = (self.D + 8) * 2.0 ** -24 * abs(scale) * torch.einsum("hd,thd->ht", q.abs(), k[seen].abs()).amax(1)
                    w = torch.softmax(s, 1)
                    out[r0] = torch.einsum("ht,thd->hd", w, v[seen])
                    lse[r0] = torch.logsumexp(s, 1)
                    mass = torch.einsum("ht,thd->hd", w, v[seen].abs())
                    run = 2 * d + (len(seen) + 64) * 2.0 ** -22
                    low = 2.0 ** -8 if self.dtype == torch.bfloat16 else 2.0 ** -24
                    tol[r0] = mass * (run[:, None] + (low if self.dtype == torch.bfloat16 else 0)) + out[r0].abs() * low
                    tol_l[r0] = run + lse[r0].abs() * 2.0 ** -23
                    r0 += 1
                begin += x
        return out, lse, tol, tol_l

    def check(self, **kw):
        out, lse = self.run(**kw)
        want, want_l, tol, tol_l = self.reference(kw.get("scale"))
        assert bool(((out.double() - want).abs() <= tol).all()), float(((out.double() - want).abs() - tol).max())
        assert bool(((lse.double() - want_l).abs() <= tol_l).all()), float(((lse.double() - want_l).abs() - tol_l).max())


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (8, 2, 128), (6, 2, 64), (16, 1, 128), (10, 2, 64), (64, 1, 64), (4, 4, 128), (32, 1, 128), (2, 2, 64)])
@pytest.mark.parametrize("page", [1, 7, 16, 64])
def test_windows(cuda_lib, dtype, Hq, Hkv, D, page):
    """Ragged windows over lengths around the tiles' and pages' edges, an empty history and an empty window among them."""
    ctx = [0, 1, 15, 16, 17, 63, 64, 65, 127, 200, 33, 0]
    lens = [[1], [3], [1], [5], [2], [1], [8], [4], [1], [2], [], []]
    Case(ctx, lens, Hq, Hkv, D, page, dtype, seed=Hq * 10 + page).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 64, 16), (4, 1, 128, 5), (3, 3, 64, 32)])
def test_candidates(cuda_lib, dtype, Hq, Hkv, D, page):
    """Block-diagonal windows: candidates of a request do not see each other, whatever their lengths."""
    ctx = [0, 70, 31, 129, 5]
    lens = [[3, 1, 4], [2, 2, 2, 2], [1], [6, 5, 9, 1, 1, 7], [20, 30]]
    Case(ctx, lens, Hq, Hkv, D, page, dtype, seed=page).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout,q_pad", [("hnd", 0), ("both", 64)])
def test_layouts_and_strides(cuda_lib, dtype, layout, q_pad):
    Case([40, 3, 100], [[4], [2, 3], [1]], 8, 4, 64, 16, dtype, seed=3, layout=layout, q_pad=q_pad).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 5, 1)])
def test_long_histories(cuda_lib, dtype, D, Hq, Hkv):
    """A few requests of long and very unlike lengths, so that each is split over the machine and joined."""
    Case([5000, 3, 777], [[2], [1], [4, 3]], Hq, Hkv, D, 16, dtype, seed=D, cands=True).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_windows(cuda_lib, dtype):
    """A prompt: windows of hundreds of rows, causal."""
    Case([0, 37], [[200], [130]], 4, 2, 64, 16, dtype, seed=5).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_peaked_rows_and_scales(cuda_lib, dtype):
    """Scores of hundreds, a scale of zero (the mean) and a negative one."""
    Case([100, 260], [[3], [1]], 4, 2, 64, 16, dtype, seed=6, heavy=True).check()
    for scale in (0.0, -0.2, 2.0):
        Case([100, 20], [[3], [2]], 4, 2, 64, 16, dtype, seed=7).check(scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale,heavy", [(None, True), (0.0, False), (-0.2, False), (2.0, False)])
def test_high_tiles_peaked_rows_and_scales(cuda_lib, D, scale, heavy):
    """Row tiles of 128: maxima that move by hundreds from tile to tile, a scale of zero and negative ones."""
    c = Case([700, 20, 333], [[3, 2], [4], [30]], 32, 1, D, 16, BF, seed=30 + D, heavy=heavy)
    # Scores that rise along the history, so that the running maximum moves at every tile.
    rise = torch.linspace(0.2, 4.0, 64)
    for b, n in enumerate((705, 24, 363)):
        for t in range(n):
            p, i = int(c.table[b, t // 16]), t % 16
            c.k[0, p, i] = (c.k[0, p, i].float() * rise[min(63, t // 12)]).to(BF)
    c.check(**({} if scale is None else {"scale": scale}))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout,q_pad,page", [("hnd", 0, 16), ("both", 64, 7), ("nhd", 0, 1), ("nhd", 0, 1000)])
def test_high_tiles_layouts(cuda_lib, D, layout, q_pad, page):
    Case([300, 0, 64, 129], [[9], [5, 4], [3, 1, 20], [17]], 48, 3, D, page, BF, seed=D + page, layout=layout, q_pad=q_pad).check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_high_tiles_split_repeats_and_bad_pages(cuda_lib, D):
    """Long requests of many stacked rows, split over the machine: the same bits every time, from a graph too; hidden pages."""
    c = Case([9000, 4000, 10], [[5], [3, 3], [2]], 64, 2, D, 16, BF, seed=40 + D)
    c.check()
    q, cache, layer, table, ctx, cu, cand = c.args
    want = api.sv_window_attention(*c.args, want_lse=True)
    for _ in range(3):
        got = api.sv_window_attention(*c.args, want_lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.sv_window_attention(*c.args, want_lse=True)
    other = api.sv_window_attention(q * 0.5, *c.args[1:], want_lse=True)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and not torch.equal(other[0], want[0])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    broken = table.clone()
    broken[1, :200] = 1 << 20
    broken[2] = -1
    got = api.sv_window_attention(q, cache, layer, broken, ctx, cu, cand, want_lse=True, status=status)
    assert int(status) == api.SV_DATA_BAD_PAGE
    assert torch.equal(got[0][:5], want[0][:5])
    assert bool((got[0][11:13] == 0).all()) and bool((got[1][11:13] == -INF).all())
    keep = torch.arange(3200, 4001)
    k = c.k[0][c.table[1].long()[keep // 16], keep % 16].double().repeat_interleave(32, 1)
    s = torch.einsum("hd,thd->ht", c.q[5].double(), k) * D ** -0.5
    assert (torch.logsumexp(s, 1) - got[1][5].cpu().double()).abs().max() < 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,rows", [(1, 3), (2, 4), (5, 3), (8, 4), (3, 40)])
def test_fp32_row_tiles(cuda_lib, D, group, rows):
    """Each height of the fp32 row tiles: maxima that move at every tile, units split over CTAs, pages that hide a part of a tile."""
    c = Case([900, 0, 64, 130], [[rows], [1, rows], [rows], [rows]], 3 * group, 3, D, 7, F32, seed=50 + D + rows, layout="both", q_pad=4)
    rise = torch.linspace(0.2, 4.0, 64)
    for t in range(900 + rows):
        p, i = int(c.table[0, t // 7]), t % 7
        c.k[0, p, i] *= rise[min(63, t // 14)]
    c.check()
    q, cache, layer, table, ctx, cu, cand = c.args
    want = api.sv_window_attention(*c.args, want_lse=True)
    broken = table.clone()
    broken[0, 3:60] = 1 << 20  # tokens 21 .. 419
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.sv_window_attention(q, cache, layer, broken, ctx, cu, cand, want_lse=True, status=status)
    assert int(status) == api.SV_DATA_BAD_PAGE
    assert torch.equal(got[0][rows:c.R - 3], want[0][rows:c.R - 3]) and torch.equal(got[1][rows:c.R - 3], want[1][rows:c.R - 3])
    at = torch.tensor([t for t in range(900 + rows) if not 21 <= t < 420])
    page = c.table[0].long()[at // 7]
    k, v = (x[0][page, at % 7].double().repeat_interleave(group, 1) for x in (c.k, c.v))
    s = torch.einsum("hd,thd->ht", c.q[rows - 1].double(), k) * D ** -0.5
    o = torch.einsum("ht,thd->hd", torch.softmax(s, 1), v)
    # A score is off by (D + 8) 2^-24 of its sum of magnitudes; a weight by twice that and the sums' (n + 64) 2^-22.
    d = (D + 8) * 2.0 ** -24 * D ** -0.5 * torch.einsum("hd,thd->ht", c.q[rows - 1].double().abs(), k.abs()).amax(1, keepdim=True)
    bound = 2 * d + (len(at) + 64) * 2.0 ** -22
    assert ((torch.logsumexp(s, 1) - got[1][rows - 1].cpu().double()).abs() <= bound[:, 0] + 1e-6).all()
    assert ((o - got[0][rows - 1].cpu().double()).abs() <= 2 * bound * v.abs().amax()).all()


@pytest.mark.gpu
def test_thousands_of_sequences(cuda_lib):
    """More sequences than a CTA has threads: every thread walks several of them."""
    gen = torch.Generator().manual_seed(3)
    ctx = torch.randint(0, 20, (3001,), generator=gen).tolist()
    Case(ctx, [[1]] * 3001, 2, 1, 64, 16, BF, seed=3, cands=False).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_requests(cuda_lib, dtype):
    """More requests than the machine has processors, most of them short."""
    gen = torch.Generator().manual_seed(9)
    ctx = torch.randint(0, 90, (400,), generator=gen).tolist()
    ctx[17], ctx[300] = 1500, 900
    lens = [[int(x)] for x in torch.randint(1, 4, (400,), generator=gen)]
    Case(ctx, lens, 4, 2, 64, 16, dtype, seed=9, cands=False).check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_many_short_units_of_high_tiles(cuda_lib, D):
    """Many stacked rows over few tokens: units of one or two key tiles, several to a share, some longer ones between them."""
    gen = torch.Generator().manual_seed(10)
    ctx = torch.randint(0, 100, (260,), generator=gen).tolist()
    ctx[100], ctx[101], ctx[200] = 700, 0, 400
    lens = [[int(x)] if x < 9 else [3, int(x)] for x in torch.randint(1, 12, (260,), generator=gen)]
    lens[7] = []
    Case(ctx, lens, 64, 4, D, 16, BF, seed=10).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_single_tokens(cuda_lib, dtype):
    """cu_draft None: one row a sequence, as with offsets of zeros."""
    c = Case([0, 5, 300, 64], [[1], [1], [1], [1]], 8, 2, 128, 16, dtype, seed=11, cands=False)
    c.check()
    q, cache, layer, table, ctx = c.args[:5]
    a = api.sv_window_attention(q, cache, layer, table, ctx, c.args[5], want_lse=True)
    b = api.sv_window_attention(q[:4], cache, layer, table, ctx, want_lse=True)
    assert torch.equal(a[0][:4], b[0]) and torch.equal(a[1][:4], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_data_errors(cuda_lib, dtype):
    """Pages out of range hide their tokens, a row that sees none gives zero and -inf; windows that do not fit are left alone."""
    c = Case([20, 40, 4], [[2], [3], [2]], 4, 2, 64, 8, dtype, seed=12)
    c.run()
    q, cache, layer, table, ctx, cu, cand = c.args
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = api.sv_window_attention(q, cache, layer, table, ctx, cu, cand, want_lse=True)
    broken = table.clone()
    broken[1, 0], broken[1, 2] = 10000, -1
    broken[2] = -1
    got = api.sv_window_attention(q, cache, layer, broken, ctx, cu, cand, want_lse=True, status=status)
    assert int(status) == api.SV_DATA_BAD_PAGE
    assert torch.equal(got[0][:2], good[0][:2])
    assert bool((got[0][5:7] == 0).all()) and bool((got[1][5:7] == -INF).all())
    # Request 1 without tokens 0..7 and 16..23.
    keep = [t for t in range(43) if t // 8 not in (0, 2)]
    k = c.k[0][c.table[1].long()[torch.tensor(keep) // 8], torch.tensor(keep) % 8].double().repeat_interleave(2, 1)
    for i in range(3):
        n = len([t for t in keep if t <= 40 + i])
        s = torch.einsum("hd,thd->ht", c.q[2 + i].double(), k[:n]) / 8
        assert (torch.logsumexp(s, 1) - got[1][2 + i].cpu().double()).abs().max() < 1e-4
    for bad_ctx, bit in ((-1, api.SV_DATA_BAD_SEQ), (1 << 30, api.SV_DATA_BAD_SEQ), (table.shape[1] * 8 - 1, api.SV_DATA_BAD_PAGE)):
        status.zero_()
        x = ctx.clone()
        x[1] = bad_ctx
        out = torch.full_like(q, 7.0)
        api.sv_window_attention(q, cache, layer, table, x, cu, cand, out=out, status=status)
        assert int(status) == bit
        assert torch.equal(out[:2], good[0][:2]) and bool((out[2:5] == 7).all()) and torch.equal(out[5:7], good[0][5:7])
    for offsets in ([0, 2, 1, 3], [0, 1, 90, 91], [-2, 1, 3, 4]):
        status.zero_()
        api.sv_window_attention(q, cache, layer, table, ctx, torch.tensor(offsets, dtype=torch.int32, device="cuda"), status=status)
        assert int(status) & api.SV_DATA_BAD_OFFSETS


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_repeats_streams_and_graphs(cuda_lib, dtype):
    """The same bits every time, on two streams at once, and from captured calls that are replayed together on new lengths."""
    c = Case([900, 30, 2000, 0], [[2], [4], [1], [3]], 8, 2, 64, 16, dtype, seed=13)
    c.run()
    q, cache, layer, table, ctx, cu, cand = c.args
    want = api.sv_window_attention(*c.args, want_lse=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [api.sv_window_attention(*c.args, want_lse=True, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)
    graphs = []
    ctxs = [ctx.clone() for _ in range(2)]
    for x in ctxs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = api.sv_window_attention(q, cache, layer, table, x, cu, cand, want_lse=True)
        graphs.append((g, o))
    ctxs[1].copy_(torch.tensor([800, 10, 100, 0], dtype=torch.int32))
    short = api.sv_window_attention(q, cache, layer, table, ctxs[1], cu, cand, want_lse=True)
    torch.cuda.synchronize()
    for (g, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1][0], want[0]) and torch.equal(graphs[1][1][0], short[0])
    assert torch.equal(graphs[0][1][1], want[1]) and torch.equal(graphs[1][1][1], short[1])


@pytest.mark.gpu
def test_offsets_past_32_bits(cuda_lib):
    """A page at the end of a pool of 6.6 GB."""
    P, page, H, D = 400, 64, 1, 128
    wide = torch.zeros(1, P, page, H, 1000 * D + D, dtype=BF, device="cuda")
    k, v = wide[..., :D], wide[..., D:2 * D]
    cache = api.KVCache(k, v)
    gen = torch.Generator().manual_seed(1)
    kk, vv, q = torch.randn(100, D, generator=gen), torch.randn(100, D, generator=gen), torch.randn(1, 2, D, generator=gen)
    table = torch.tensor([[P - 1, P - 2]], dtype=torch.int32, device="cuda")
    for i, p in ((0, P - 1), (1, P - 2)):
        n = min(64, 100 - 64 * i)
        k[0, p, :n, 0], v[0, p, :n, 0] = kk[64 * i:64 * i + n].cuda().to(BF), vv[64 * i:64 * i + n].cuda().to(BF)
    ctx = torch.tensor([99], dtype=torch.int32, device="cuda")
    out, _ = api.sv_window_attention(q.to(BF).cuda(), cache, 0, table, ctx)
    s = torch.softmax(q.to(BF).double()[0] @ kk.to(BF).double().T * D ** -0.5, 1)
    assert (out.cpu().double()[0] - s @ vv.to(BF).double()).abs().max() < 0.02


@pytest.mark.gpu
def test_a_step_of_all_calls(cuda_lib):
    """Two steps of a small model with four candidates a request: reserve, append and attention for both layers, verify, select,
    log probabilities, commit. The cache then holds what the kept tokens' rows were, and a step with the kept candidate alone
    gives the same attention."""
    torch.manual_seed(3)
    B, n, K, H, D, V, L, page = 5, 4, 3, 2, 64, 512, 2, 8
    dev = "cuda"
    k = torch.full((L, 64, page, H, D), float("nan"), dtype=BF, device=dev)
    cache = api.KVCache(k, k.clone())
    table = torch.full((B, 8), -1, dtype=torch.int32, device=dev)
    ctx = torch.zeros(B, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    rows = K + 1
    cu = torch.arange(0, B * n * K + 1, K, dtype=torch.int32, device=dev)
    cand = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=dev)
    R = B * n * rows
    wo = torch.randn(2 * H * D, V, device=dev) * 0.2
    held = [[] for _ in range(B)]  # the kept rows' keys, in order
    for step in range(2):
        lo = ctx.clone()
        assert bool((api.sv_cache_reserve(cache, table, ctx, cu, cand, status=status) == n * rows).all())
        new = torch.randn(L, R, H, D, device=dev).to(BF)
        q = torch.randn(L, R, 2 * H, D, device=dev).to(BF)
        outs = []
        for layer in range(L):
            api.sv_cache_append(cache, layer, new[layer], -new[layer], table, ctx, cu, cand, status=status)
            outs.append(api.sv_window_attention(q[layer], cache, layer, table, ctx, cu, cand, status=status)[0])
        logits = (outs[-1].view(R, -1).float() @ wo).contiguous()
        tokens = torch.randint(0, V, (B * n * K,), dtype=torch.int32, device=dev)
        pick = torch.rand(B * n * K, device=dev) < 0.7
        target = logits.view(B * n, rows, V)[:, :K].argmax(2).view(-1).to(torch.int32)
        tokens = torch.where(pick, target, tokens)
        out_tokens, out_len = api.spec_verify_greedy(logits, tokens, cu)
        u = torch.rand(B, device=dev)
        best, best_len = api.sv_select_candidates(cand, out_len, api.SV_SELECT_UNIFORM, u)
        lp = api.sv_token_logprobs(logits, out_tokens, cu_draft=cu, out_len=out_len, n_top=1, status=status)
        for c in range(B * n):  # greedy commits are the rows' first choices
            at = slice(c * rows, c * rows + int(out_len[c]))
            assert bool((lp.rank[at] == 1).all()) and torch.equal(lp.top_ids[at, 0], out_tokens[at])
        api.sv_cache_commit(cache, table, ctx, cu, out_len, cand, best, status=status)
        assert torch.equal(ctx, lo + best_len) and int(status) == 0
        for b in range(B):
            r0 = int(best[b]) * rows
            held[b] += [new[:, r] for r in range(r0, r0 + int(best_len[b]))]
            for t, x in enumerate(held[b]):
                p = int(table[b, t // page])
                assert torch.equal(cache.k[:, p, t % page], x) and torch.equal(cache.v[:, p, t % page], -x)
            assert int((table[b] >= 0).sum()) == -(-len(held[b]) // page)


@pytest.mark.gpu
def test_two_threads_on_one_stream(cuda_lib):
    """Calls of two host threads on the same stream and cache, each with its own windows, all of them split and joined."""
    import threading
    c = Case([9000, 700, 3000], [[3], [2], [1]], 8, 2, 64, 16, BF, seed=21)
    c.run()
    q, cache, layer, table, ctx, cu, cand = c.args
    short = torch.tensor([100, 650, 3000], dtype=torch.int32, device="cuda")
    args = [c.args, (-q, cache, layer, table, short, cu, cand)]
    want = [api.sv_window_attention(*a, want_lse=True) for a in args]
    torch.cuda.synchronize()
    got, start = [[], []], threading.Barrier(2)

    def work(i):
        start.wait()
        for _ in range(200):
            got[i].append(api.sv_window_attention(*args[i], want_lse=True))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 200
        assert all(torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1]) for g in got[i])


@pytest.mark.gpu
def test_dimensions_of_one_take_no_step(cuda_lib):
    """One head, one row, one layer: their strides may be anything, as torch leaves them behind a transpose or a slice."""
    c = Case([30, 7], [[2], [1]], 1, 1, 64, 16, BF, seed=4, cands=False)
    c.check()
    q, cache, layer, table, ctx, cu = c.args[:6]
    want = api.sv_window_attention(q, cache, 0, table, ctx, cu)[0]
    odd, out = (torch.empty(1, c.R, 64, dtype=BF, device="cuda").transpose(0, 1) for _ in range(2))  # [R, 1, D] of [1, R, D]
    odd.copy_(q)
    assert odd.stride(1) != 64 and odd.is_contiguous()
    assert torch.equal(api.sv_window_attention(odd, cache, 0, table, ctx, cu)[0], want)
    api.sv_window_attention(odd, cache, 0, table, ctx, cu, out=out)
    assert torch.equal(out[:3], want[:3])
    # Keys of one head, and a single row whose keys and values come from buffers of other widths.
    k = torch.zeros(1, 6, 4, 1, 64, dtype=BF, device="cuda")
    cache = api.KVCache(k, k.clone())
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.sv_cache_reserve(cache, table, ctx)
    wide_k, wide_v = torch.randn(1, 1, 128, device="cuda").to(BF), torch.randn(1, 1, 192, device="cuda").to(BF)
    api.sv_cache_append(cache, 0, wide_k[..., :64], wide_v[..., 64:128], table, ctx)
    assert torch.equal(cache.k[0, 0, 0], wide_k[0, :, :64]) and torch.equal(cache.v[0, 0, 0], wide_v[0, :, 64:128])
    # A cache of one layer whose K and V lie in buffers of different depth.
    a, b = (torch.zeros(*s, 4, 1, 64, dtype=BF, device="cuda") for s in ((2, 6), (6, 1)))
    b = b.transpose(0, 1)
    assert a[:1].stride() != b.stride()
    cache = api.KVCache(a[:1], b, cache.page_ref, cache.free_bits)  # the page is held
    api.sv_cache_append(cache, 0, wide_k[..., :64], wide_v[..., 64:128], table, ctx)
    assert torch.equal(a[0, 0, 0], wide_k[0, :, :64]) and torch.equal(b[0, 0, 0], wide_v[0, :, 64:128])
    with pytest.raises(ValueError):
        api.sv_window_attention(q.expand(-1, 2, -1), cache, 0, table, ctx, cu)
