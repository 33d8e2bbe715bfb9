"""The page operations (sv_cache_*) against the same operations on host
lists, their refusals (CPU) and their data errors."""
import ctypes
import os
import random
import subprocess
import sys

import pytest
import torch

from cache_model import Model
from speculative_decoding_verification_27_gb300 import api, build

FAKE = 0x10000  # never dereferenced: validation rejects first
ODD = 0x10001


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return api.load()


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE, dtype=1, n_layers=2, n_pages=10, page_size=4, n_kv_heads=2, head_dim=64, layer_stride=5120,
             page_stride=512, token_stride=128, head_stride=64, page_ref=FAKE, free_bits=FAKE)
    a.update(kw)
    return ctypes.byref(api._Cache(*a.values()))


def _seqs(**kw):
    a = dict(table=FAKE, table_stride=8, table_pages=8, n=3, ctx_len=FAKE)
    a.update(kw)
    return ctypes.byref(api._Sequences(*a.values()))


def _calls(lib):
    """Every call of the family with good arguments, any of them replaced."""
    def fork(cache=None, seqs=None, N=2, src=FAKE, dst=FAKE, status=None):
        return lib.sv_cache_fork(cache or _cache(), seqs or _seqs(), N, src, dst, status, None)

    def free(cache=None, seqs=None, N=2, which=FAKE, status=None):
        return lib.sv_cache_free(cache or _cache(), seqs or _seqs(), N, which, status, None)

    def reserve(cache=None, seqs=None, n_cand=3, cu=FAKE, cand=None, granted=None, ws=FAKE, wsb=1 << 20, status=None):
        return lib.sv_cache_reserve(cache or _cache(), seqs or _seqs(), n_cand, cu, cand, granted, ws, wsb, status, None)

    def append(cache=None, layer=0, n_layers=2, k=FAKE, v=FAKE, ls=1280, rs=128, R=10, seqs=None, n_cand=3, cu=FAKE, cand=None,
               status=None):
        return lib.sv_cache_append(cache or _cache(), layer, n_layers, k, v, ls, rs, R, seqs or _seqs(), n_cand, cu, cand,
                                   status, None)

    def commit(cache=None, seqs=None, n_cand=3, cu=FAKE, cand=None, best=None, n=FAKE, status=None):
        return lib.sv_cache_commit(cache or _cache(), seqs or _seqs(), n_cand, cu, cand, best, n, status, None)

    return fork, free, reserve, append, commit


def test_host_validation_of_the_descriptions(lib):
    E = api.SV_ERR_INVALID_ARG
    bad_caches = [dict(k=0), dict(v=0), dict(k=FAKE + 8), dict(dtype=2), dict(n_layers=0), dict(n_pages=0), dict(page_size=0),
                  dict(n_kv_heads=0), dict(head_dim=0), dict(head_dim=60), dict(layer_stride=4), dict(page_stride=-8),
                  dict(token_stride=129), dict(head_stride=1 << 62), dict(page_ref=0), dict(page_ref=ODD), dict(free_bits=0),
                  dict(free_bits=ODD)]
    bad_seqs = [dict(table=0), dict(table=ODD), dict(table_stride=7), dict(table_pages=0), dict(n=-1), dict(ctx_len=0),
                dict(ctx_len=ODD)]
    for call in _calls(lib):
        for c in bad_caches:
            assert call(cache=_cache(**c)) == E, (call, c)
        for s in bad_seqs:
            assert call(seqs=_seqs(**s)) == E, (call, s)
        assert call(status=ODD) == E


def test_host_validation_of_the_calls(lib):
    E, OK = api.SV_ERR_INVALID_ARG, api.SV_OK
    fork, free, reserve, append, commit = _calls(lib)
    assert fork(N=0) == OK and free(N=0) == OK and append(R=0) == OK and append(n_layers=0) == OK
    empty = _seqs(n=0, table=0, ctx_len=0)
    for call in (reserve, append, commit):
        assert call(seqs=empty, n_cand=0) == OK
        assert call(n_cand=-1) == E and call(n_cand=2) == E and call(cu=ODD) == E
        assert call(cu=None, cand=FAKE) == E and call(cand=ODD) == E
    for bad in (dict(N=-1), dict(src=None), dict(dst=None), dict(src=ODD), dict(dst=ODD)):
        assert fork(**bad) == E
    for bad in (dict(N=-1), dict(which=None), dict(which=ODD)):
        assert free(**bad) == E
    for bad in (dict(ws=None), dict(ws=FAKE + 8), dict(wsb=16 + 3 * 16 - 1), dict(granted=ODD),
                dict(seqs=_seqs(n=16385), n_cand=16385)):
        assert reserve(**bad) == E
    for bad in (dict(layer=-1), dict(layer=1), dict(n_layers=-1), dict(n_layers=3), dict(k=None), dict(v=None), dict(k=FAKE + 8),
                dict(ls=4), dict(rs=4), dict(rs=-128), dict(R=-1)):
        assert append(**bad) == E
    for bad in (dict(n=None), dict(n=ODD), dict(best=FAKE), dict(cand=FAKE), dict(cand=FAKE, best=ODD)):
        assert commit(**bad) == E
    assert lib.sv_cache_reserve_workspace_size(3) == 64
    assert lib.sv_cache_reserve_workspace_size(-1) == 0 and lib.sv_cache_reserve_workspace_size(16385) == 0


def test_binding_refuses(lib):
    k = torch.zeros(1, 4, 2, 1, 64)
    with pytest.raises(ValueError):
        api.KVCache(k, k)


# ---------------------------------------------------------------------------
# On the GPU
# ---------------------------------------------------------------------------
def _value(name, L, H, D, dtype):
    """A token's keys, one row a (layer, head): its name in two digits, the layer and the head, all exact in bf16."""
    x = torch.zeros(L, H, D)
    x[..., 0], x[..., 1] = name % 256, name // 256
    x[..., 2] = torch.arange(L)[:, None]
    x[..., D - 1] = torch.arange(H)[None]
    return x.to(dtype)


class Rig:
    """A cache on the GPU and its model, driven together."""

    def __init__(self, n=12, width=9, n_pages=70, page=7, L=2, H=2, D=64, dtype=torch.bfloat16, layout="nhd"):
        self.m = Model(n_pages, page, n, width)
        self.L, self.H, self.D, self.dtype = L, H, D, dtype
        shape = (L, n_pages, page, H, D)
        if layout == "nhd":
            k, v = (torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        elif layout == "hnd":
            k, v = (torch.full((L, n_pages, H, page, D), float("nan"), dtype=dtype, device="cuda").transpose(2, 3)
                    for _ in range(2))
        else:  # K and V of a page together, and a gap behind every token
            both = torch.full((n_pages, L, 2, page, H, D + 16), float("nan"), dtype=dtype, device="cuda")[..., :D]
            k, v = both[:, :, 0].transpose(0, 1), both[:, :, 1].transpose(0, 1)
        self.cache = api.KVCache(k, v)
        buf = torch.full((n, width + 3), -7, dtype=torch.int32, device="cuda")
        self.table = buf[:, :width]
        self.table.fill_(-1)
        self.ctx = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.names = 0

    def args(self):
        return self.cache, self.table, self.ctx

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def bits(self):
        b = int(self.status)
        self.status.zero_()
        return b

    def check(self):
        m = self.m
        assert self.table.cpu().tolist() == m.table
        assert self.ctx.cpu().tolist() == m.ctx
        assert self.cache.page_ref.cpu().tolist() == m.ref
        assert [x % (1 << 32) for x in self.cache.free_bits.cpu().tolist()] == m.free_words()
        k, v = self.cache.k.cpu(), self.cache.v.cpu()
        for b in range(len(m.ctx)):
            for t, name in enumerate(m.tokens(b)):
                p, i = m.table[b][t // m.P], t % m.P
                want = _value(name, self.L, self.H, self.D, self.dtype)
                assert torch.equal(k[:, p, i], want), (b, t)
                assert torch.equal(v[:, p, i], want * 2), (b, t)

    def step(self, rng, cands=None):
        """One step of the loop for every sequence: windows of random candidates, one kept."""
        m, n = self.m, len(self.m.ctx)
        lens = [[rng.randint(1, 5) for _ in range(1 if cands is None else rng.choice(cands))] for _ in range(n)]
        cu, cand = [0], [0]
        for x in lens:
            for y in x:
                cu.append(cu[-1] + y - 1)
            cand.append(cand[-1] + len(x))
        g_cu, g_cand = self.i32(cu), None if cands is None else self.i32(cand)
        rows = [sum(x) for x in lens]
        granted = api.sv_cache_reserve(*self.args(), g_cu, g_cand, status=self.status)
        want, short, wide = m.reserve(rows)
        assert granted.cpu().tolist() == want
        assert self.bits() == (api.SV_DATA_NO_PAGES if short else 0) | (api.SV_DATA_BAD_PAGE if wide else 0)
        names = [list(range(self.names + sum(rows[:b]), self.names + sum(rows[:b + 1]))) for b in range(n)]
        self.names += sum(rows)
        flat = [x for y in names for x in y]
        new = torch.stack([_value(x, self.L, self.H, self.D, self.dtype) for x in flat], 1).cuda() if flat else \
            torch.zeros(self.L, 0, self.H, self.D, dtype=self.dtype, device="cuda")
        api.sv_cache_append(self.cache, 0, new[:1], new[:1] * 2, self.table, self.ctx, g_cu, g_cand, status=self.status)
        for layer in range(1, self.L):
            api.sv_cache_append(self.cache, layer, new[layer], new[layer] * 2, self.table, self.ctx, g_cu, g_cand)
        # A window without room: rows that found no page are flagged and skipped; what room there was may be written.
        refused = [b for b in range(n) if rows[b] and not want[b]]
        assert self.bits() in ((0, api.SV_DATA_BAD_PAGE) if refused else (0,))
        m.append(names, want)
        best, out, kept = [], [0] * (len(cu) - 1), []
        for b in range(n):
            i = rng.randrange(len(lens[b])) if lens[b] else -1
            if i < 0 or not want[b]:
                best.append(-1 if cands is not None else b)
                kept.append((0, 0))
                continue
            c = cand[b] + i
            out[c] = rng.randint(0, lens[b][i])
            best.append(c)
            kept.append((sum(lens[b][:i]), out[c]))
        api.sv_cache_commit(*self.args(), g_cu, self.i32(out), g_cand, None if cands is None else self.i32(best),
                            status=self.status)
        m.commit(kept)
        assert self.bits() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("page,layout,dtype,H,D,cands", [
    (7, "nhd", torch.bfloat16, 2, 64, None), (1, "hnd", torch.float32, 1, 64, [0, 1, 2, 4]), (16, "both", torch.bfloat16, 3, 128, [1, 3]),
    (4, "nhd", torch.float32, 5, 8, [1, 2]), (64, "hnd", torch.bfloat16, 8, 128, [4])])
def test_random_steps(cuda_lib, page, layout, dtype, H, D, cands):
    """Forks, steps and ends in a random order, on a pool that runs short at times."""
    rng = random.Random(page * 100 + D)
    r = Rig(page=page, layout=layout, dtype=dtype, H=H, D=D, width=max(3, 40 // page), n_pages=max(20, 300 // page), L=3)
    n = len(r.m.ctx)
    short = False
    for _ in range(25):
        r.step(rng, cands)
        r.check()
        if rng.random() < 0.4:
            which = [rng.randrange(n) for _ in range(rng.randint(0, 4))]  # repeats among them
            api.sv_cache_free(*r.args(), r.i32(which), status=r.status)
            r.m.free(which)
            assert r.bits() == 0
        empty = [b for b in range(n) if not r.m.ctx[b]]
        live = [b for b in range(n) if r.m.ctx[b]]
        if empty and live:
            dst = rng.sample(empty, rng.randint(1, len(empty)))
            src = [rng.choice(live) for _ in dst]
            api.sv_cache_fork(*r.args(), r.i32(src), r.i32(dst), status=r.status)
            assert not r.m.fork(src, dst) and r.bits() == 0
        r.check()
    api.sv_cache_free(*r.args(), r.i32(list(range(n))))
    r.m.free(range(n))
    r.check()
    assert r.m.ref == [0] * r.m.n_pages and not short


@pytest.mark.gpu
def test_sharers_of_one_partial_page(cuda_lib):
    """Five holders of one partly filled page reserve in one call: four copies, the last keeps it; with one holder outside the
    call, five copies; when pages run out between them, the later sharers get nothing."""
    for outside in (False, True):
        for pages in (40, 9):
            r = Rig(n=8, page=8, n_pages=pages)
            one = [1] + [0] * 7
            # 13 tokens in sequence 0.
            for size in (8, 5):
                rows = [size * x for x in one]
                lens = [max(0, x - 1) for x in rows]
                cand = [0]
                for x in rows:
                    cand.append(cand[-1] + (x > 0))
                cu = [0, rows[0] - 1]
                g, cc = r.i32(cu), r.i32(cand)
                api.sv_cache_reserve(*r.args(), g, cc)
                want, _, _ = r.m.reserve(rows)
                names = [list(range(r.names, r.names + rows[0]))] + [[]] * 7
                r.names += rows[0]
                new = torch.stack([_value(x, r.L, r.H, r.D, r.dtype) for x in names[0]], 1).cuda()
                api.sv_cache_append(r.cache, 0, new, new * 2, r.table, r.ctx, g, cc)
                r.m.append(names, want)
                api.sv_cache_commit(*r.args(), g, r.i32([rows[0]]), cc, r.i32([0] + [-1] * 7))
                r.m.commit([(0, rows[0])] + [(0, 0)] * 7)
            r.check()
            src, dst = [0] * (5 if outside else 4), [2, 3, 5, 7, 6][: 5 if outside else 4]
            api.sv_cache_fork(*r.args(), r.i32(src), r.i32(dst), status=r.status)
            assert not r.m.fork(src, dst)
            rows = [2 if b in (0, 2, 3, 5, 7) else 0 for b in range(8)]
            cand, cu = [0], [0]
            for x in rows:
                cand.append(cand[-1] + (x > 0))
                if x:
                    cu.append(cu[-1] + x - 1)
            granted = api.sv_cache_reserve(*r.args(), r.i32(cu), r.i32(cand), status=r.status)
            want, short, _ = r.m.reserve(rows)
            assert granted.cpu().tolist() == want
            assert r.bits() == (api.SV_DATA_NO_PAGES if short else 0)
            r.check()


@pytest.mark.gpu
def test_reserve_twice_and_cancel(cuda_lib):
    """A second reserve uses what the first one took; a commit of nothing and an end both give it back."""
    r = Rig(page=4, n=3, n_pages=20)
    for rows in ([3, 9, 0], [6, 2, 1]):
        cu = [0]
        for x in rows:
            cu.append(cu[-1] + max(x, 1) - 1)
        cand = [0]
        for x in rows:
            cand.append(cand[-1] + (x > 0))
        cu2 = [0]
        for x in rows:
            if x:
                cu2.append(cu2[-1] + x - 1)
        api.sv_cache_reserve(*r.args(), r.i32(cu2), r.i32(cand), status=r.status)
        r.m.reserve(rows)
        r.check()
    api.sv_cache_commit(*r.args(), r.i32(cu2), r.i32([0] * (len(cu2) - 1)), r.i32(cand), r.i32([0, 1, 2]), status=r.status)
    r.m.commit([(0, 0)] * 3)
    r.check()
    assert r.m.ref == [0] * 20
    api.sv_cache_reserve(*r.args(), r.i32([0, 0, 2, 4]))
    r.m.reserve([1, 3, 3])
    api.sv_cache_free(*r.args(), r.i32([0, 1, 2]))
    r.m.free([0, 1, 2])
    r.check()
    assert r.bits() == 0


@pytest.mark.gpu
def test_one_row_a_sequence(cuda_lib):
    """Without offsets every sequence has a window of one row."""
    r = Rig(page=2, n=4, n_pages=30)
    for step in range(5):
        assert api.sv_cache_reserve(*r.args()).cpu().tolist() == [1] * 4
        r.m.reserve([1] * 4)
        names = [[r.names + b] for b in range(4)]
        r.names += 4
        new = torch.stack([_value(x[0], r.L, r.H, r.D, r.dtype) for x in names], 1).cuda()
        api.sv_cache_append(r.cache, 0, new, new * 2, r.table, r.ctx)
        r.m.append(names, [1] * 4)
        keep = [1, 1, step % 2, 1]
        api.sv_cache_commit(*r.args(), None, r.i32(keep), status=r.status)
        r.m.commit([(0, x) for x in keep])
        r.check()
    assert r.bits() == 0


@pytest.mark.gpu
def test_data_errors_leave_the_rest_alone(cuda_lib):
    rng = random.Random(4)
    r = Rig(page=4, n=6, n_pages=60)
    r.step(rng)
    r.check()
    live = [b for b in range(6) if r.m.ctx[b]]
    # fork: a taken destination, an index out of range, a destination twice, a source that is a destination
    r.m.free([5, 4])
    api.sv_cache_free(*r.args(), r.i32([5, 4, 5]))
    for src, dst in (([live[0]], [live[1]]), ([-1], [5]), ([0], [6]), ([99], [5]), ([0, 1], [5, 5]), ([0, 4], [4, 5])):
        api.sv_cache_fork(*r.args(), r.i32(src), r.i32(dst), status=r.status)
        assert r.m.fork(src, dst)
        assert r.bits() == api.SV_DATA_BAD_SEQ, (src, dst)
        r.check()
        r.m.free([4, 5])
        api.sv_cache_free(*r.args(), r.i32([4, 5]))
        r.check()
    api.sv_cache_free(*r.args(), r.i32([6, -1]), status=r.status)
    assert r.bits() == api.SV_DATA_BAD_SEQ
    r.check()
    # windows: offsets that decrease, a negative offset, candidates out of range
    for cu, cand in (([0, 2, 1, 3, 4, 5, 6], None), ([-1, 0, 1, 2, 3, 4, 5], None), ([0, 1, 2], [0, 1, 2, 3, 3, 3, 3]),
                     ([0, 1, 2], [0, 1, 0, 2, 2, 2, 2]), ([0, 1, 2], [-1, 1, 2, 2, 2, 2, 2])):
        before = [x.clone() for x in (r.table, r.ctx, r.cache.page_ref, r.cache.free_bits)]
        one = 1 if cand else len(cu) - 1
        api.sv_cache_commit(*r.args(), r.i32(cu), r.i32([0] * (len(cu) - 1)), None if cand is None else r.i32(cand),
                            None if cand is None else r.i32([-1] * 6), status=r.status)
        assert r.bits() & api.SV_DATA_BAD_OFFSETS, (cu, cand, one)
        assert all(torch.equal(a, b) for a, b in zip(before, (r.table, r.ctx, r.cache.page_ref, r.cache.free_bits)))
    # commit: more rows than the candidate has, a candidate of another request, rows without pages
    ones = r.i32([0, 1, 2, 3, 4, 5, 6])
    for n, best in (([3, 0, 0, 0, 0, 0], None), ([0, 0, -1, 0, 0, 0], None)):
        api.sv_cache_commit(*r.args(), ones, r.i32(n), status=r.status)
        assert r.bits() == api.SV_DATA_BAD_OFFSETS
        r.check()
    api.sv_cache_commit(*r.args(), ones, r.i32([0] * 6), r.i32(list(range(7))), r.i32([0, 2, 2, 3, 4, 5]), status=r.status)
    assert r.bits() == api.SV_DATA_BAD_OFFSETS
    r.check()
    api.sv_cache_commit(*r.args(), ones, r.i32([0, 0, 0, 0, 0, 2]), status=r.status)
    assert r.bits() == api.SV_DATA_BAD_PAGE
    r.check()
    # lengths and pages out of range in the tables
    for what, value, bit in (("ctx", -3, api.SV_DATA_BAD_SEQ), ("ctx", 1 << 30, api.SV_DATA_BAD_SEQ)):
        keep = r.ctx.clone()
        r.ctx[live[0]] = value
        assert api.sv_cache_reserve(*r.args(), ones, status=r.status)[live[0]] == 0
        assert r.bits() == bit
        r.m.reserve([2 if b != live[0] else 0 for b in range(6)])
        r.ctx.copy_(keep)
        r.check()
    b = live[0]
    page = int(r.table[b, 0])
    for wrong in (60, 1 << 30):
        r.table[b, 0] = wrong
        ref = r.cache.page_ref.clone()
        api.sv_cache_fork(*r.args(), r.i32([b]), r.i32([5]), status=r.status)
        assert r.bits() in (api.SV_DATA_BAD_PAGE, api.SV_DATA_BAD_SEQ) and torch.equal(ref, r.cache.page_ref)
        new = torch.zeros(12, r.H, r.D, dtype=r.dtype, device="cuda")
        api.sv_cache_append(r.cache, 0, new, new, r.table[b:b + 1], torch.zeros(1, dtype=torch.int32, device="cuda"), status=r.status)
        assert r.bits() == api.SV_DATA_BAD_PAGE
    r.table[b, 0] = page
    r.check()


@pytest.mark.gpu
def test_offsets_past_32_bits(cuda_lib):
    """Pages whose elements lie more than 2^32 into the pool, in every layer."""
    L, P, page, H, D = 2, 20000, 64, 8, 128
    wide = torch.empty(L, P, page, H, 2, D, dtype=torch.bfloat16, device="cuda")[..., 1, :]  # 10.5 GB of each
    v = torch.empty(L, P, page, H, 2, D, dtype=torch.bfloat16, device="cuda")[..., 1, :]
    ref = torch.ones(P, dtype=torch.int32, device="cuda")
    bits = torch.zeros(-(-P // 32), dtype=torch.int32, device="cuda")
    for p in (P - 1, P - 2, P - 5):
        ref[p] = 0
        bits[p // 32] |= 1 << p % 32
    cache = api.KVCache(wide, v, ref, bits)
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(2, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 39, 79], dtype=torch.int32, device="cuda")
    assert api.sv_cache_reserve(cache, table, ctx, cu).tolist() == [40, 41]
    assert table[:, 0].tolist() == [P - 5, P - 2] and table[:, 1].tolist() == [-1, -1]
    new = torch.randn(L, 81, H, D, device="cuda").bfloat16()
    api.sv_cache_append(cache, 0, new, -new, table, ctx, cu)
    api.sv_cache_commit(cache, table, ctx, cu, torch.tensor([40, 0], dtype=torch.int32, device="cuda"))
    assert ctx.tolist() == [40, 0] and table[:, 0].tolist() == [P - 5, -1]
    api.sv_cache_fork(cache, table, ctx, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"))
    assert api.sv_cache_reserve(cache, table, ctx).tolist() == [1, 1]
    assert table[:, 0].tolist() == [P - 2, P - 5]
    for p in (P - 5, P - 2):
        assert torch.equal(wide[:, p, :40], new[:, :40]) and torch.equal(v[:, p, :40], -new[:, :40])


@pytest.mark.gpu
def test_free_pages_far_into_a_large_pool(cuda_lib):
    """More pages than one sweep of the allocator covers, free ones here and there; bits past the last page do not count."""
    P = 100003
    k = torch.zeros(1, P, 1, 1, 8, device="cuda")
    free = sorted(random.Random(2).sample(range(40000, P), 50)) + [P - 1]
    ref = torch.ones(P, dtype=torch.int32)
    words = [0] * -(-P // 32)
    for p in free:
        ref[p] = 0
        words[p // 32] |= 1 << p % 32
    bits = torch.tensor([w - (1 << 32) if w >> 31 else w for w in words], dtype=torch.int32, device="cuda")
    bits[-1] |= 1 << 30  # stray bits behind the last page
    assert P % 32 < 30
    cache = api.KVCache(k, k.clone(), ref.cuda(), bits)
    table = torch.full((60, 3), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(60, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.sv_cache_reserve(cache, table, ctx, status=status).cpu()
    assert int(status) == api.SV_DATA_NO_PAGES and got.tolist() == [1] * 51 + [0] * 9
    assert table[:51, 0].cpu().tolist() == sorted(set(free)) and int((cache.page_ref != 1).sum()) == 0


@pytest.mark.gpu
def test_append_from_a_wider_projection(cuda_lib):
    """k_new and v_new as slices of one projection's output: rows with a stride."""
    r = Rig(page=4, n=3, n_pages=20, H=2, D=64)
    cu = r.i32([0, 2, 2, 5])
    api.sv_cache_reserve(*r.args(), cu)
    qkv = torch.randn(8, 3, 2, 64, device="cuda").to(r.dtype)
    for layer in range(r.L):
        api.sv_cache_append(r.cache, layer, qkv[:, 1], qkv[:, 2], r.table, r.ctx, cu, status=r.status)
    assert r.bits() == 0
    row = 0
    for b, n in enumerate((3, 1, 4)):
        for t in range(n):
            p = int(r.table[b, t // 4])
            for layer in range(r.L):
                assert torch.equal(r.cache.k[layer, p, t % 4], qkv[row, 1]) and torch.equal(r.cache.v[layer, p, t % 4], qkv[row, 2])
            row += 1
    with pytest.raises(ValueError):
        api.sv_cache_append(r.cache, 0, qkv[:, 1], qkv[:, 2].contiguous(), r.table, r.ctx, cu)
    with pytest.raises(ValueError):
        api.sv_cache_append(r.cache, 0, qkv[:, 1].float(), qkv[:, 2].float(), r.table, r.ctx, cu)


@pytest.mark.gpu
def test_largest_batch_of_reserve(cuda_lib):
    n = api.SV_CACHE_MAX_SEQS
    k = torch.zeros(1, n + 40, 2, 1, 8, device="cuda")
    cache = api.KVCache(k, k.clone())
    table = torch.full((n, 2), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert bool((api.sv_cache_reserve(cache, table, ctx, status=status) == 1).all())
    assert torch.equal(table[:, 0].cpu(), torch.arange(n, dtype=torch.int32)) and int(status) == 0
    ctx.fill_(2)  # full pages: each of the next windows needs one more, of which 40 are left
    got = api.sv_cache_reserve(cache, table, ctx, status=status).cpu()
    assert int(got.sum()) == 40 and bool((got[:40] == 1).all()) and int(status) == api.SV_DATA_NO_PAGES
    assert int((cache.page_ref == 0).sum()) == 0 and int(cache.free_bits.abs().sum()) == 0


@pytest.mark.gpu
def test_a_captured_step(cuda_lib):
    """reserve, append and commit captured once and replayed: lengths and tables move on by themselves."""
    r = Rig(page=4, n=3, n_pages=40, width=12)
    new = torch.zeros(r.L, 9, r.H, r.D, dtype=r.dtype, device="cuda")
    twice = new * 2
    cu, n = r.i32([0, 2, 4, 6]), r.i32([0, 0, 0])

    from_host = torch.zeros_like(n)

    def step():
        n.copy_(from_host)  # a copy node before the kernels
        api.sv_cache_reserve(*r.args(), cu)
        api.sv_cache_append(r.cache, 0, new, twice, r.table, r.ctx, cu)
        api.sv_cache_commit(*r.args(), cu, n)

    step()
    r.m.reserve([3] * 3)
    r.m.commit([(0, 0)] * 3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for keep in ([3, 1, 2], [1, 3, 2], [2, 2, 0], [3, 3, 3]):
        names = [list(range(r.names + 3 * b, r.names + 3 * b + 3)) for b in range(3)]
        r.names += 9
        new.copy_(torch.stack([_value(x, r.L, r.H, r.D, r.dtype) for y in names for x in y], 1))
        twice.copy_(new * 2)
        from_host.copy_(r.i32(keep))
        graph.replay()
        granted, _, _ = r.m.reserve([3] * 3)
        r.m.append(names, granted)
        r.m.commit([(0, x) for x in keep])
        r.check()


_BATCHES = """
import torch
from speculative_decoding_verification_27_gb300 import api
k = torch.zeros(1, 4096, 2, 1, 8, device="cuda")
for n in (3399, 3400, 4095, 4096):
    cache = api.KVCache(k, k.clone())
    table = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
    got = api.sv_cache_reserve(cache, table, torch.zeros(n, dtype=torch.int32, device="cuda"))
    assert bool((got == 1).all()) and table[:, 0].tolist() == list(range(n)), n
print("all granted")
"""


@pytest.mark.gpu
def test_batches_around_the_default_shared_memory(cuda_lib):
    """The largest batches that fit the shared memory a kernel has without asking, and the next ones, in a process of their own: a
    larger batch before them would ask for all."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", _BATCHES], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "all granted" in p.stdout, p.stderr[-2000:]


@pytest.mark.gpu
def test_a_launch_that_fails_leaves_no_error(cuda_lib):
    """Calls on a stream whose capture has become invalid report it, and leave nothing for the next one to find."""
    from test_logprobs import _logits
    rt = ctypes.CDLL("libcudart.so.13")
    stream = ctypes.c_void_p()
    r = Rig(n=2, page=4, n_pages=9)
    new = torch.zeros(r.L, 2, r.H, r.D, dtype=r.dtype, device="cuda")
    z, tok = (x.cuda() for x in _logits(2, 100, torch.float32, 1))
    one = r.i32([0])
    torch.cuda.synchronize()

    class S:  # what the binding takes of a stream
        cuda_stream = 0

    assert rt.cudaStreamCreateWithFlags(ctypes.byref(stream), 1) == 0
    S.cuda_stream = stream.value
    q = torch.zeros(2, r.H, r.D, dtype=r.dtype, device="cuda")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    granted = r.i32([0, 0])
    outs = api.sv_token_logprobs(z, tok)
    torch.cuda.synchronize()
    calls = [lambda: api.sv_cache_free(*r.args(), one, stream=S), lambda: api.sv_cache_fork(*r.args(), one, r.i32([1]), stream=S),
             lambda: api.sv_cache_reserve(*r.args(), granted=granted, workspace=ws, stream=S),
             lambda: api.sv_cache_append(r.cache, 0, new, new, r.table, r.ctx, stream=S),
             lambda: api.sv_cache_commit(*r.args(), None, granted, stream=S),
             lambda: api.sv_window_attention(q, r.cache, 0, r.table, r.ctx, out=q, workspace=ws, stream=S),
             lambda: api.sv_token_logprobs(z, tok, out_logprob=outs.logprob, out_rank=outs.rank, out_entropy=outs.entropy, stream=S)]
    rt.cudaStreamBeginCapture.argtypes = [ctypes.c_void_p, ctypes.c_int]
    rt.cudaStreamSynchronize.argtypes = [ctypes.c_void_p]
    rt.cudaStreamEndCapture.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    rt.cudaStreamDestroy.argtypes = [ctypes.c_void_p]
    left = []
    try:
        for call in calls:
            graph = ctypes.c_void_p()
            assert rt.cudaStreamBeginCapture(stream, 2) == 0  # relaxed: nothing else is affected
            assert rt.cudaStreamSynchronize(stream) != 0      # not allowed meanwhile: the capture is invalid from here on
            rt.cudaGetLastError()
            with pytest.raises(api.SpecVerifyError):
                call()
            left.append(rt.cudaGetLastError())
            rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
            rt.cudaGetLastError()
    finally:
        rt.cudaStreamDestroy(stream)
    assert left == [0] * len(calls)
    assert api.sv_cache_reserve(*r.args()).tolist() == [1, 1]


@pytest.mark.gpu
def test_candidates_whose_offsets_decrease(cuda_lib):
    """Offsets that decrease inside a request are found by every call, which leaves that request alone and serves the others."""
    r = Rig(n=3, page=4, n_pages=30, width=6)
    r.ctx.copy_(r.i32([3, 2, 0]))
    r.table[:, 0] = r.i32([0, 1, -1])
    r.cache.page_ref[:2] = 1
    r.cache.free_bits[0] &= ~3
    cand, good, bad = r.i32([0, 1, 4, 5]), r.i32([0, 1, 4, 5, 6, 8]), r.i32([0, 1, 4, 3, 6, 8])
    R = 13
    state = lambda: [x.clone() for x in (r.table, r.ctx, r.cache.page_ref)]  # noqa: E731
    before = state()
    granted = api.sv_cache_reserve(*r.args(), bad, cand, status=r.status)
    assert granted.tolist() == [2, 0, 3] and r.bits() == api.SV_DATA_BAD_OFFSETS
    assert all(torch.equal(a[1:2], b[1:2]) for a, b in zip(before[:2], state()[:2]))
    assert api.sv_cache_reserve(*r.args(), good, cand, status=r.status).tolist() == [2, 8, 3] and r.bits() == 0
    r.cache.k.zero_()
    r.cache.v.zero_()
    new = torch.ones(r.L, R, r.H, r.D, dtype=r.dtype, device="cuda")
    api.sv_cache_append(r.cache, 0, new, new, r.table, r.ctx, bad, cand, status=r.status)
    assert r.bits() == api.SV_DATA_BAD_OFFSETS
    row = r.table[1, :3].long()
    assert bool((r.cache.k[:, row] == 0).all()) and bool((r.cache.v[:, row] == 0).all())
    assert int((r.cache.k[0, :, :, 0, 0] == 1).sum()) == 5  # the rows of the other two
    q = torch.ones(R, 2 * r.H, r.D, dtype=r.dtype, device="cuda")
    out = torch.full_like(q, 7.0)
    api.sv_window_attention(q, r.cache, 0, r.table, r.ctx, bad, cand, out=out, status=r.status)
    assert r.bits() == api.SV_DATA_BAD_OFFSETS
    assert bool((out[2:10] == 7).all()) and not bool((out[:2] == 7).any()) and not bool((out[10:13] == 7).any())
    before = state()
    api.sv_cache_commit(*r.args(), bad, r.i32([1, 2, 0, 2, 1]), cand, r.i32([0, 3, 4]), status=r.status)
    assert r.bits() == api.SV_DATA_BAD_OFFSETS
    after = state()
    assert after[1].tolist() == [4, 2, 1] and torch.equal(before[0][1], after[0][1])
    api.sv_cache_commit(*r.args(), good, r.i32([0, 3, 0, 0, 0]), cand, r.i32([0, 1, 4]), status=r.status)
    assert r.bits() == 0 and r.ctx.tolist() == [4, 5, 1]


@pytest.mark.gpu
def test_fork_of_a_page_without_holders(cuda_lib):
    """A table whose page the counts call free is not forked: nothing of it is written, and the page stays what it was."""
    rng = random.Random(8)
    r = Rig(page=4, n=4, n_pages=30)
    r.step(rng)
    r.step(rng)
    r.m.free([2, 3])
    api.sv_cache_free(*r.args(), r.i32([2, 3]))
    r.check()
    b = max((0, 1), key=lambda x: r.m.ctx[x])
    assert r.m.ctx[b] > 0
    page = r.m.table[b][r.m.pages(r.m.ctx[b]) - 1]
    for count in (0, -1):
        r.cache.page_ref[page] = count
        before = [x.clone() for x in (r.table, r.ctx, r.cache.page_ref, r.cache.free_bits)]
        api.sv_cache_fork(*r.args(), r.i32([b, b]), r.i32([2, 3]), status=r.status)
        assert r.bits() == api.SV_DATA_BAD_PAGE
        assert all(torch.equal(x, y) for x, y in zip(before, (r.table, r.ctx, r.cache.page_ref, r.cache.free_bits)))
    r.cache.page_ref[page] = 1
    api.sv_cache_fork(*r.args(), r.i32([b, b]), r.i32([2, 3]), status=r.status)
    assert not r.m.fork([b, b], [2, 3]) and r.bits() == 0
    r.check()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3])
def test_append_of_the_longest_list_of_rows(cuda_lib, n):
    """R may be any int32: here one row that stands for all of them, of which the windows take a few."""
    r = Rig(n=n, page=4, n_pages=9)
    cu = r.i32([2 * b for b in range(n + 1)])
    api.sv_cache_reserve(*r.args(), cu)
    new = torch.randn(1, 1, r.H, r.D, device="cuda").to(r.dtype).expand(1, 2 ** 31 - 1, r.H, r.D)
    api.sv_cache_append(r.cache, 1, new, new, r.table, r.ctx, cu, status=r.status)
    assert r.bits() == 0
    for b in range(n):
        assert torch.equal(r.cache.k[1, int(r.table[b, 0]), :3], new[0, :3]) and torch.equal(r.cache.v[1, int(r.table[b, 0]), :3], new[0, :3])


@pytest.mark.gpu
@pytest.mark.parametrize("page,n_pages,cands", [(7, 20, None), (1, 60, [0, 1, 2, 4]), (16, 12, [1, 3]), (4, 30, [1, 2])])
def test_random_steps_that_run_short(cuda_lib, page, n_pages, cands):
    """Random steps, forks and ends on a pool that has too few pages for many of them; requests that share a partly filled page are
    refused among them."""
    rng = random.Random(page)
    r = Rig(page=page, n_pages=n_pages, width=max(3, 60 // page), L=2)
    n, plain, seen = len(r.m.ctx), r.m.reserve, []

    def reserve(rows):
        held = [r.m.table[b][r.m.ctx[b] // page] for b in range(n) if rows[b] and r.m.ctx[b] % page]
        shared = {p for p in held if r.m.ref[p] > 1}
        parts = [r.m.table[b][r.m.ctx[b] // page] if r.m.ctx[b] % page else -1 for b in range(n)]
        granted, short, wide = plain(rows)
        seen.append((short, any(rows[b] and not granted[b] and parts[b] in shared for b in range(n))))
        return granted, short, wide

    r.m.reserve = reserve
    for _ in range(30):
        r.step(rng, cands)
        if rng.random() < 0.5:
            which = rng.sample(range(n), rng.randint(1, 4))
            api.sv_cache_free(*r.args(), r.i32(which), status=r.status)
            r.m.free(which)
            assert r.bits() == 0
        empty, live = [b for b in range(n) if not r.m.ctx[b]], [b for b in range(n) if r.m.ctx[b]]
        if empty and live:
            dst = rng.sample(empty, rng.randint(1, len(empty)))
            src = [rng.choice(live) for _ in dst]
            api.sv_cache_fork(*r.args(), r.i32(src), r.i32(dst), status=r.status)
            assert not r.m.fork(src, dst) and r.bits() == 0
        r.check()
    assert sum(s for s, _ in seen) >= 5 and (page == 1 or any(x for _, x in seen))
