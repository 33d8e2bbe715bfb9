"""Caches of 8 bits as they are written and moved, and sv_rope_append, against
their definitions in 64 bits; their refusals (CPU) and data errors."""
import ctypes
import math
import random

import pytest
import torch

import test_cache
from test_cache import FAKE, ODD, Rig, _seqs, _value
from speculative_decoding_verification_27_gb300 import api, build

BF, F32, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return api.load()


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE, dtype=3, n_layers=2, n_pages=10, page_size=4, n_kv_heads=2, head_dim=64, layer_stride=5120,
             page_stride=512, token_stride=128, head_stride=64, page_ref=FAKE, free_bits=FAKE, ks=FAKE, vs=FAKE, sl=80, sp=8, st=1, sh=4)
    a.update(kw)
    return ctypes.byref(api._Cache(*a.values()))


def test_host_validation_of_scales(lib):
    E = api.SV_ERR_INVALID_ARG
    bad = [dict(ks=0), dict(vs=0), dict(ks=ODD), dict(vs=ODD), dict(sl=-1), dict(sp=1 << 62), dict(head_dim=272, head_stride=272),
           dict(head_dim=72), dict(token_stride=136), dict(dtype=4)]
    for call in test_cache._calls(lib):
        for c in bad:
            assert call(cache=_cache(**c)) == E, (call, c)
    append = test_cache._calls(lib)[3]
    assert append(cache=_cache(), ls=1284) == E and append(cache=_cache(), R=0) == api.SV_OK
    assert append(cache=_cache(dtype=1, ks=0, vs=0, sl=-1), R=0) == api.SV_OK  # scales of the other caches are not read
    # No other call takes the type of a cache.
    assert lib.sv_token_logprobs(FAKE, 3, 128, 128, 2, FAKE, 0, None, None, 1.0, 0, FAKE, FAKE, None, None, None, None, None) == E


def _rope(lib, **kw):
    r = dict(cos_sin=FAKE, stride=64, n_pos=100, rot=64, pairs=0, eps=1e-6, gq=FAKE, gk=FAKE, pos=None)
    a = dict(cache=_cache(), layer=0, rope=None, q=FAKE, qs=256, heads=4, out=FAKE, os=256, k=FAKE, v=FAKE, rs=128, R=10, seqs=_seqs(),
             n_cand=3, cu=FAKE, cand=None, status=None)
    for x, y in kw.items():
        (r if x in r else a)[x] = y
    if a["rope"] is None:
        a["rope"] = ctypes.byref(api._Rope(*r.values()))
    elif a["rope"] == "null":
        a["rope"] = None
    return lib.sv_rope_append(*a.values(), None)


def test_host_validation_of_rope(lib):
    E, OK = api.SV_ERR_INVALID_ARG, api.SV_OK
    assert _rope(lib, R=0) == OK and _rope(lib, seqs=_seqs(n=0), n_cand=0) == OK
    assert _rope(lib, R=0, rot=0, cos_sin=None) == OK and _rope(lib, R=0, gq=None, gk=None, eps=0.0) == OK
    wide = dict(token_stride=1 << 12, page_stride=1 << 14, layer_stride=1 << 20)
    for bad in (dict(rope="null"), dict(layer=-1), dict(layer=2), dict(heads=0), dict(q=None), dict(q=FAKE + 8), dict(out=None),
                dict(out=FAKE + 8), dict(k=None), dict(v=FAKE + 8), dict(qs=255), dict(qs=260), dict(qs=128), dict(os=128), dict(os=260),
                dict(rs=4), dict(rs=-128), dict(R=-1), dict(n_cand=2), dict(cand=ODD), dict(cu=None, cand=FAKE), dict(cu=ODD),
                dict(status=ODD), dict(cos_sin=None), dict(cos_sin=FAKE + 4), dict(stride=48), dict(stride=66), dict(n_pos=-1), dict(rot=-16),
                dict(rot=24), dict(rot=80), dict(pairs=2), dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf), dict(eps=-1.0),
                dict(gq=FAKE + 8), dict(gk=ODD), dict(pos=ODD), dict(cache=_cache(ks=0)),
                dict(cache=_cache(dtype=0, head_dim=260, head_stride=260, **wide)), dict(cache=_cache(dtype=0, head_dim=60, head_stride=60, **wide))):
        assert _rope(lib, **bad) == E, bad


def test_rope_in_place_has_one_stride(lib):
    E, OK = api.SV_ERR_INVALID_ARG, api.SV_OK
    assert _rope(lib, qs=256, os=264) == E and _rope(lib, qs=264, os=256) == E
    assert _rope(lib, qs=256, os=264, R=0) == OK


def test_appends_write_no_common_scales(lib):
    """Scales that several places share (strides of zero) may be read by attention, not written row by row."""
    E, OK = api.SV_ERR_INVALID_ARG, api.SV_OK
    calls = test_cache._calls(lib)
    one = dict(n_layers=1, n_pages=1, page_size=1, n_kv_heads=1)
    for c, size in ((dict(sl=0), "n_layers"), (dict(sp=0), "n_pages"), (dict(st=0), "page_size"), (dict(sh=0), "n_kv_heads")):
        assert calls[3](cache=_cache(**c), R=0) == E and _rope(lib, cache=_cache(**c), R=0) == E
        alone = _cache(**{**one, **c})
        assert calls[3](cache=alone, n_layers=1, R=0) == OK and _rope(lib, cache=alone, R=0) == OK, size
        assert lib.sv_window_attention(FAKE, 256, 4, 0, _cache(**c), 0, _seqs(), 3, FAKE, None, 0.1, FAKE, 256, None, FAKE, 1 << 30, None, None) == OK


def test_rope_as_bytes():
    """The binding packs the description as the library reads it."""
    want = bytes(api._Rope(0x1230, 64, 100, 48, 1, 1e-5, 0x4560, 0x7890, 0xabc0))
    assert api._pack_rope(0x1230, 64, 100, 48, True, 1e-5, 0x4560, 0x7890, 0xabc0) == want


# ---------------------------------------------------------------------------
# A cache of 8 bits
# ---------------------------------------------------------------------------
def quantised(x):
    """(e4m3 values, scales) of rows along the last dimension by the definition, in fp32 on the host. (A quotient of two tensors:
    a number over a tensor is that number times a rounded reciprocal.)"""
    most = x.float().abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
    return (x.float() * (torch.full_like(most, 448.0) / most)).to(E8), (most / 448.0)[..., 0]


def cache8(L, P, page, H, D, layout):
    """An empty cache whose places hold what no append writes: NaN values, scales of NaN."""
    raw = lambda *s: torch.full(s, 0x7F, dtype=torch.uint8, device="cuda")  # noqa: E731
    nan = lambda *s: torch.full(s, math.nan, device="cuda")  # noqa: E731
    if layout == "nhd":
        k, v = raw(L, P, page, H, D), raw(L, P, page, H, D)
        ks, vs = nan(L, P, page, H), nan(L, P, page, H)
    elif layout == "hnd":
        k, v = (raw(L, P, H, page, D).transpose(2, 3) for _ in range(2))
        ks, vs = (nan(L, P, H, page).transpose(2, 3) for _ in range(2))
    else:  # K and V of a page together, with gaps
        both = raw(P, L, 2, page, H, D + 32)[..., :D]
        k, v = both[:, :, 0].transpose(0, 1), both[:, :, 1].transpose(0, 1)
        pair = nan(P, page, L, H, 2)
        ks, vs = (pair[..., i].permute(2, 0, 1, 3) for i in range(2))
    return api.KVCache(k.view(E8), v.view(E8), k_scale=ks, v_scale=vs)


class Rig8(Rig):
    """The page operations' rig on a cache of 8 bits: rows by name are bf16, as appended."""

    def __init__(self, layout="nhd", n_pages=70, page=7, L=2, H=2, D=64, **kw):
        super().__init__(n_pages=n_pages, page=page, L=L, H=H, D=D, **kw)
        self.cache = cache8(L, n_pages, page, H, D, layout)

    def check(self):
        m = self.m
        assert self.table.cpu().tolist() == m.table and self.ctx.cpu().tolist() == m.ctx
        assert self.cache.page_ref.cpu().tolist() == m.ref
        c = self.cache
        k, v = c.k.view(torch.uint8).cpu(), c.v.view(torch.uint8).cpu()
        ks, vs = c.k_scale.cpu(), c.v_scale.cpu()
        for b in range(len(m.ctx)):
            for t, name in enumerate(m.tokens(b)):
                p, i = m.table[b][t // m.P], t % m.P
                x = _value(name, self.L, self.H, self.D, BF)
                for rows, raw, scale in ((x, k, ks), (x * 2, v, vs)):
                    want, want_scale = quantised(rows)
                    assert torch.equal(raw[:, p, i], want.view(torch.uint8)), (b, t)
                    assert torch.equal(scale[:, p, i], want_scale), (b, t)


@pytest.mark.gpu
@pytest.mark.parametrize("page,layout,H,D,cands", [(7, "nhd", 2, 64, None), (1, "hnd", 1, 128, [0, 1, 2, 4]), (16, "both", 3, 256, [1, 3]),
                                                    (4, "hnd", 5, 16, [1, 2]), (64, "both", 8, 80, [4])])
def test_random_steps_in_8_bits(cuda_lib, page, layout, H, D, cands):
    """Forks, steps with kept candidates and ends: values and their scales are where the page tables say."""
    rng = random.Random(page * 100 + D)
    r = Rig8(page=page, layout=layout, H=H, D=D, width=max(3, 40 // page), n_pages=max(20, 300 // page), L=3)
    n = len(r.m.ctx)
    for _ in range(12):
        r.step(rng, cands)
        r.check()
        which = [rng.randrange(n) for _ in range(rng.randint(0, 3))]
        api.sv_cache_free(*r.args(), r.i32(which), status=r.status)
        r.m.free(which)
        empty, live = [b for b in range(n) if not r.m.ctx[b]], [b for b in range(n) if r.m.ctx[b]]
        if empty and live:
            dst = rng.sample(empty, rng.randint(1, len(empty)))
            src = [rng.choice(live) for _ in dst]
            api.sv_cache_fork(*r.args(), r.i32(src), r.i32(dst), status=r.status)
            r.m.fork(src, dst)
        assert r.bits() == 0
        r.check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 64, 128, 144, 256])
def test_quantised_rows(cuda_lib, D):
    """Rows of every magnitude, zeros and single values among them, against the definition's bound: half a step of three bits of
    fraction (2^-4 of the value; 2^-10 scales below the smallest normal value), and two roundings in fp32."""
    gen = torch.Generator().manual_seed(D)
    R, H = 333, 3
    x = torch.randn(R, H, 2 * D, generator=gen) * torch.exp2(torch.randint(-90, 120, (R, H, 1), generator=gen).float())
    x[5], x[6, :, 3:], x[7] = 0.0, 0.0, 3e38
    x[8], x[9] = x[8] * 2.0 ** -130, 1.0
    x = x.to(BF)
    c = cache8(1, R, 1, H, D, "nhd")
    table = torch.full((1, R), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, R - 1], dtype=torch.int32, device="cuda")
    api.sv_cache_reserve(c, table, ctx, cu)
    g = x.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.sv_cache_append(c, 0, g[..., :D].contiguous(), g[..., D:].contiguous(), table, ctx, cu, status=status)
    assert int(status) == 0
    p = table[0].long().cpu()
    for rows, pool, scale in ((x[..., :D], c.k, c.k_scale), (x[..., D:], c.v, c.v_scale)):
        q, s = pool.view(torch.uint8).cpu()[0, p, 0].view(E8), scale.cpu()[0, p, 0]
        want, want_s = quantised(rows)
        assert torch.equal(q.view(torch.uint8), want.view(torch.uint8)) and torch.equal(s, want_s)
        back, exact = q.double() * s.double()[..., None], rows.double()
        assert bool(((back - exact).abs() <= exact.abs() * (2.0 ** -4 + 2.0 ** -21) + s.double()[..., None] * 2.0 ** -10).all())


# ---------------------------------------------------------------------------
# Norm, rotation and append in one pass
# ---------------------------------------------------------------------------
def turned(x, pos, g, table, pairs, eps):
    """The definition in 64 bits, and how far fp32 may be from it: a norm's sum of D squares is off by D 2^-24 of itself, its root
    and the products after it by a few roundings, and every turned element by two roundings of its two terms."""
    D, x = x.shape[-1], x.double()
    rel = 4 * 2.0 ** -24
    if g is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * g.double()
        rel += (D / 2 + 8) * 2.0 ** -24
    off = x.abs()
    if table is not None:
        rot, half = table.shape[1], table.shape[1] // 2
        c, s = table[pos].double()[:, None].split(half, 2)
        pick = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, half), slice(half, rot))
        u, w = x[..., pick[0]], x[..., pick[1]]
        x, off = x.clone(), off.clone()
        x[..., pick[0]], x[..., pick[1]] = u * c - w * s, w * c + u * s
        off[..., pick[0]], off[..., pick[1]] = (u * c).abs() + (w * s).abs(), (w * c).abs() + (u * s).abs()
    return x, rel * off


class RopeCase:
    def __init__(self, ctx, lens, Hq, Hkv, D, page, dtype, rot, pairs=False, norm=(True, True), seed=0, layout="nhd", cands=True):
        gen = torch.Generator().manual_seed(seed)
        self.__dict__.update(ctx=ctx, lens=lens, D=D, page=page, dtype=dtype, pairs=pairs, Hq=Hq, Hkv=Hkv)
        row = BF if dtype == E8 else dtype
        n = len(ctx)
        rows = [sum(y) for y in lens]
        self.R = sum(rows) + 3
        P = sum(-(-(c + r) // page) for c, r in zip(ctx, rows)) + 2
        if dtype == E8:
            self.cache = cache8(2, P, page, Hkv, D, layout)
        else:
            k, v = (torch.full((2, P, page, Hkv, D), math.nan, dtype=row, device="cuda") for _ in range(2))
            if layout == "hnd":
                k, v = (x.transpose(2, 3).contiguous().transpose(2, 3) for x in (k, v))
            self.cache = api.KVCache(k, v)
        self.table = torch.full((n, max(-(-(c + r) // page) for c, r in zip(ctx, rows)) + 1), -1, dtype=torch.int32, device="cuda")
        zero = torch.zeros(n, dtype=torch.int32, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        cu, cand = [0], [0]
        for y in lens:
            cand.append(cand[-1] + len(y))
            for x in y:
                cu.append(cu[-1] + x - 1)
        lots = [c + r for c, r in zip(ctx, rows)]
        # A window of all tokens reserves the pages (a sequence without any has no candidate).
        api.sv_cache_reserve(self.cache, self.table, zero, i32([0] + [sum(x - 1 for x in lots[:i + 1] if x) for i in range(n) if lots[i]]),
                             i32([0] + [sum(1 for x in lots[:i + 1] if x) for i in range(n)]))
        self.ctx_len = i32(ctx)
        self.cu, self.cand = i32(cu), i32(cand) if cands else None
        self.both = (torch.randn(self.R, (Hq + 2 * Hkv) * D, generator=gen) * 3.0).to(row)
        self.g = [(1 + 0.3 * torch.randn(D, generator=gen)).to(row) if x else None for x in norm]
        n_pos = max(ctx) + max(max(y, default=0) for y in lens) + 1
        angle = torch.arange(n_pos)[:, None].double() * 10000.0 ** (-torch.arange(0, rot, 2).double() / max(rot, 1))
        self.cs = torch.cat([angle.cos(), angle.sin()], 1).float() if rot else None

    def split(self, both):
        q, k, v = both.split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], 1)
        return q.view(self.R, self.Hq, self.D), k.view(self.R, self.Hkv, self.D), v.view(self.R, self.Hkv, self.D)

    def run(self, layer=1, positions=None, in_place=False, **kw):
        q, k, v = self.split(self.both.cuda())
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = q if in_place else torch.full((self.R, self.Hq, self.D), 7.0, dtype=q.dtype, device="cuda")
        dev = lambda x: None if x is None else x.cuda()  # noqa: E731
        self.args = (q, k, v, self.cache, layer, self.table, self.ctx_len, self.cu, self.cand)
        self.kw = dict(cos_sin=dev(self.cs), q_norm=dev(self.g[0]), k_norm=dev(self.g[1]), eps=1e-5, pairs=self.pairs, positions=dev(positions))
        api.sv_rope_append(*self.args, **self.kw, out=out, status=status, **kw)
        return out.cpu(), int(status)

    def check(self, layer=1, positions=None, **kw):
        out, status = self.run(layer, positions, **kw)
        assert status == 0
        q, k, v = self.split(self.both)
        low = torch.finfo(q.dtype).eps / 2
        r0, c = 0, self.cache
        table = self.table.cpu().long()
        left = torch.ones(self.R, dtype=torch.bool)
        k8 = [x.view(torch.uint8).cpu() if self.dtype == E8 else x.cpu() for x in (c.k, c.v)]
        scales = [x.cpu() for x in (c.k_scale, c.v_scale)] if self.dtype == E8 else [None, None]
        for b, y in enumerate(self.lens):
            n = sum(y)
            rows, t = slice(r0, r0 + n), self.ctx[b] + torch.arange(n)
            left[rows] = False
            pos = self.ctx[b] + torch.cat([torch.arange(x) for x in y]) if y else t
            if positions is not None:
                pos = positions[rows].long()
            want, tol = turned(q[rows], pos, self.g[0], self.cs, self.pairs, 1e-5)
            assert bool(((out[rows].double() - want).abs() <= tol + (want.abs() + tol) * low).all())
            at = (layer, table[b, t // self.page], t % self.page)
            for x, g, pool, scale in ((k, self.g[1], k8[0], scales[0]), (v, None, k8[1], scales[1])):
                want, tol = turned(x[rows], pos, g, self.cs, self.pairs, 1e-5) if x is k else (x[rows].double(), torch.zeros(1).double())
                got = (pool[at] if scale is None else pool[at].view(E8)).double()
                if scale is None:
                    assert bool(((got - want).abs() <= (tol + (want.abs() + tol) * low if x is k else 0.0)).all())
                    continue
                s = scale[at].double()
                most = want.abs().amax(2) / 448
                assert bool(((s - most).abs() <= tol.amax(-1) / 448 + most * 2.0 ** -23).all())
                s = s[..., None]
                assert bool(((got * s - want).abs() <= tol + (want.abs() + tol) * (2.0 ** -4 + 2.0 ** -21) + s * 2.0 ** -10).all())
            r0 += n
        kept = q if kw.get("in_place") else torch.full_like(out, 7.0)
        assert torch.equal(out[left], kept[left])
        other = c.k[1 - layer].float() if self.dtype != E8 else c.k_scale[1 - layer]
        assert bool(other.isnan().all())  # the other layer is untouched


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32, E8])
@pytest.mark.parametrize("Hq,Hkv,D,page,rot,pairs,norm", [
    (8, 2, 128, 16, 128, False, (True, True)), (4, 4, 64, 7, 32, True, (False, False)), (1, 1, 64, 1, 64, False, (True, False)),
    (12, 3, 128, 5, 64, True, (False, True)), (3, 1, 256, 16, 256, False, (True, True)), (5, 5, 80, 4, 48, False, (True, True)),
    (2, 1, 16, 3, 16, True, (True, True)), (6, 2, 144, 8, 0, False, (True, True)), (32, 8, 128, 16, 128, True, (True, True))])
def test_rope_append(cuda_lib, dtype, Hq, Hkv, D, page, rot, pairs, norm):
    """Ragged windows with candidates, an empty history, a sequence without a window and long ones."""
    ctx = [0, 1, 15, 130, 33, 64, 0]
    lens = [[1], [3, 2, 4], [1], [70], [], [5, 1, 1, 9], [33]]
    RopeCase(ctx, lens, Hq, Hkv, D, page, dtype, rot, pairs, norm, seed=D + Hq, layout="hnd" if Hq == 12 else "nhd").check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32, E8])
def test_rope_positions_and_in_place(cuda_lib, dtype):
    """Positions of the caller's, and queries rotated where they are."""
    c = RopeCase([100, 4], [[3, 2], [6]], 6, 2, 64, 8, dtype, 64, seed=2)
    c.check(positions=torch.tensor([9, 0, 103, 77, 5, 1, 1, 2, 3, 103, 50, -7, 1 << 30, 0], dtype=torch.int32))
    RopeCase([100, 4], [[3, 2], [6]], 6, 2, 64, 8, dtype, 32, seed=3).check(in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,rot,pairs", [(64, 32, False), (64, 16, True), (80, 48, False), (128, 64, True), (256, 32, False)])
def test_rope_keeps_what_is_not_turned(cuda_lib, dtype, D, rot, pairs):
    """Without norms an infinity or a NaN behind the turned elements is its element's own: every other one keeps its bits."""
    got = []
    for special in (False, True):
        c = RopeCase([33, 4], [[3, 2], [6]], 6, 2, D, 8, dtype, rot, pairs, (False, False), seed=D)
        x = c.both.view(c.R, -1, D)
        put = torch.zeros_like(x, dtype=torch.bool)
        for r in range(c.R):
            put[r, r % 8, rot + r % (D - rot)] = put[r, (r + 3) % 8, rot + 5 * r % (D - rot)] = True
        if special:
            x[put] = torch.tensor([math.inf, -math.inf, math.nan], dtype=x.dtype).repeat(c.R)[: int(put.sum())]
        out, status = c.run()
        assert status == 0
        got.append((c, out, put, x))
    (a, out_a, put, _), (b, out_b, _, x) = got
    q, k, v = (y.transpose(0, 1) for y in x.transpose(0, 1).split([6, 2, 2]))
    rows = slice(0, 11)
    assert torch.equal(out_a[rows][~put[rows, :6]], out_b[rows][~put[rows, :6]])
    assert torch.equal(out_b[rows][put[rows, :6]].nan_to_num(3.5), q[rows][put[rows, :6]].nan_to_num(3.5))
    table, r0 = b.table.cpu().long(), 0
    for s, n in ((0, 5), (1, 6)):
        t = b.ctx[s] + torch.arange(n)
        at, now = (1, table[s, t // 8], t % 8), slice(r0, r0 + n)
        for pool, rows, h in (("k", k, 6), ("v", v, 8)):
            x0, x1, special = getattr(a.cache, pool).cpu()[at], getattr(b.cache, pool).cpu()[at], put[now, h: h + 2]
            assert torch.equal(x0[~special], x1[~special])
            assert torch.equal(x1[special].nan_to_num(3.5), rows[now][special].nan_to_num(3.5))
        r0 += n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32, E8])
def test_rope_single_rows_and_many_sequences(cuda_lib, dtype):
    """cu_draft of None, a row a sequence, and more rows than warps."""
    ctx = torch.randint(0, 60, (700,), generator=torch.Generator().manual_seed(1)).tolist()
    c = RopeCase(ctx, [[1]] * 700, 4, 2, 64, 8, dtype, 64, seed=4, cands=False)
    c.check()
    a = api.sv_rope_append(*c.args, **c.kw)
    b = api.sv_rope_append(*(x[:700] for x in c.args[:3]), *c.args[3:7], **c.kw)
    assert torch.equal(a[:700], b) and not bool(a[700:].any())
    RopeCase([5, 9], [[2500], [900]], 8, 2, 128, 16, dtype, 128, seed=5, cands=False).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, E8])
def test_rope_data_errors(cuda_lib, dtype):
    """Positions off the table leave a row out; windows without a page of their own still get their queries; windows that do not
    fit are left alone."""
    c = RopeCase([20, 30, 4], [[2], [3], [2]], 4, 2, 64, 8, dtype, 64, seed=6, cands=False)
    good, _ = c.run(layer=0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    raw = lambda: (c.cache.k.view(torch.uint8) if dtype == E8 else c.cache.k.view(torch.int16)).clone()  # noqa: E731
    before = raw()
    out = torch.full_like(c.args[0], 7.0)
    pos = torch.tensor([20, -1, 33, 33, 32, 4, 33 + 1, 0, 0, 0], dtype=torch.int32, device="cuda")  # the table has 34 rows
    api.sv_rope_append(*c.args[:4], 1, *c.args[5:], **{**c.kw, "positions": pos}, out=out, status=status)
    assert int(status) == api.SV_DATA_BAD_POSITION
    assert [bool((out[r] == 7).all()) for r in range(10)] == [False, True, False, False, False, False, True, True, True, True]
    after = raw()
    table = c.table.cpu()
    for b, t, kept in ((0, 20, 0), (0, 21, 1), (1, 30, 0), (2, 4, 0), (2, 5, 1)):
        p = int(table[b, t // 8])
        assert torch.equal(before[1, p, t % 8], after[1, p, t % 8]) == bool(kept)
    # A page out of range, one that is shared, none.
    status.zero_()
    broken = c.table.clone()
    broken[0, 2], broken[1, 3] = 1 << 20, -1
    c.cache.page_ref[int(table[2, 0])] = 2
    out = torch.full_like(c.args[0], 7.0)
    (c.cache.k.view(torch.uint8) if dtype == E8 else c.cache.k.view(torch.int16))[1] = 0x7F
    before = raw()
    api.sv_rope_append(*c.args[:4], 1, broken, *c.args[6:], **c.kw, out=out, status=status)
    assert int(status) == api.SV_DATA_BAD_PAGE and torch.equal(out[:7].cpu(), good[:7])
    written = (raw() != before).flatten(3).any(3)[1].nonzero().tolist()
    assert written == [[int(table[1, 4]), 0]]  # token 32 of request 1 alone
    c.cache.page_ref[int(table[2, 0])] = 1
    for bad, bit in ((-1, api.SV_DATA_BAD_SEQ), (1 << 30, api.SV_DATA_BAD_SEQ)):
        status.zero_()
        x = c.ctx_len.clone()
        x[1] = bad
        out = torch.full_like(c.args[0], 7.0)
        api.sv_rope_append(*c.args[:6], x, *c.args[7:], **c.kw, out=out, status=status)
        assert int(status) == bit
        assert torch.equal(out[:2].cpu(), good[:2]) and bool((out[2:5] == 7).all()) and torch.equal(out[5:7].cpu(), good[5:7])
    status.zero_()
    api.sv_rope_append(*c.args[:7], torch.tensor([0, 1, 90, 91], dtype=torch.int32, device="cuda"), **c.kw, status=status)
    assert int(status) & api.SV_DATA_BAD_OFFSETS


@pytest.mark.gpu
def test_rope_captured_and_on_another_stream(cuda_lib):
    """A captured call replays on new lengths and rows; a call on a stream of the caller's gives the same bits."""
    c = RopeCase([40, 9, 0], [[2], [3], [4]], 8, 2, 128, 16, E8, 128, seed=8, cands=False)
    want, _ = c.run()
    args = list(c.args)
    args[6] = c.ctx_len.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.sv_rope_append(*args, **c.kw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:9].cpu(), want[:9])
    args[6].copy_(torch.tensor([38, 10, 0], dtype=torch.int32))
    args[0].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    fresh = api.sv_rope_append(*args, **c.kw)
    assert torch.equal(out, fresh) and not torch.equal(out[:9].cpu(), want[:9])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = api.sv_rope_append(*args, **c.kw, stream=s)
    s.synchronize()
    assert torch.equal(other, fresh)


@pytest.mark.gpu
def test_binding_of_rope_refuses(cuda_lib):
    c = RopeCase([4], [[2]], 4, 2, 64, 8, BF, 64, seed=9, cands=False)
    c.run()
    q, k, v = c.args[:3]
    for bad in ((q.float(), k, v), (q[:, :, :32], k, v), (q, k[:2], v), (q, k, v.float()), (q, k, v.contiguous()), (q.transpose(1, 2), k, v)):
        with pytest.raises(ValueError):
            api.sv_rope_append(*bad, *c.args[3:], **c.kw)
    for bad in (dict(cos_sin=c.kw["cos_sin"].double()), dict(cos_sin=c.kw["cos_sin"].cpu()), dict(q_norm=c.kw["q_norm"].float()),
                dict(k_norm=c.kw["k_norm"][:32]), dict(positions=torch.zeros(c.R, dtype=torch.int64, device="cuda")),
                dict(positions=torch.zeros(c.R - 1, dtype=torch.int32, device="cuda")), dict(out=torch.zeros_like(q).float())):
        with pytest.raises(ValueError):
            api.sv_rope_append(*c.args, **{**c.kw, **bad})
    with pytest.raises(api.SpecVerifyError):
        api.sv_rope_append(*c.args, **{**c.kw, "cos_sin": c.kw["cos_sin"][:, :24]})
    k8 = torch.zeros(1, 4, 2, 1, 64, device="cuda").to(E8)
    ks = torch.ones(1, 4, 2, 1, device="cuda")
    for bad in (dict(k_scale=ks), dict(k_scale=ks, v_scale=ks.double()), dict(k_scale=ks, v_scale=ks[:, :2]), dict(k_scale=ks.cpu(), v_scale=ks)):
        with pytest.raises(ValueError):
            api.KVCache(k8, k8, **bad)
    with pytest.raises(ValueError):
        api.KVCache(k8.to(BF), k8.to(BF), k_scale=ks, v_scale=ks)
    assert api.KVCache(k8, k8.clone()).k_scale.shape == (1, 4, 2, 1)
