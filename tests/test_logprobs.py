"""sv_token_logprobs: log probability, rank, entropy and top alternatives of
rows of logits, against their definition in 64 bits; the refusals of the
entry point (CPU) and the data errors."""
import ctypes
import math

import pytest
import torch

from speculative_decoding_verification_27_gb300 import api, build

FAKE = ctypes.c_void_p(0x10000)       # never dereferenced: validation rejects first
MISALIGNED = ctypes.c_void_p(0x10001)
INF = math.inf


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return api.load()


def _call(lib, **kw):
    a = dict(z=FAKE, dt=1, V=100, ld=100, R=4, tok=FAKE, B=0, cu=None, ln=None, T=1.0, n=5, lp=FAKE, rank=FAKE, ent=FAKE,
             ids=FAKE, tlp=FAKE, st=FAKE)
    a.update(kw)
    return lib.sv_token_logprobs(a["z"], a["dt"], a["V"], a["ld"], a["R"], a["tok"], a["B"], a["cu"], a["ln"], a["T"], a["n"],
                                 a["lp"], a["rank"], a["ent"], a["ids"], a["tlp"], a["st"], None)


def test_host_validation(lib):
    E = api.SV_ERR_INVALID_ARG
    assert _call(lib, R=0) == api.SV_OK
    assert _call(lib, B=0, cu=FAKE, ln=FAKE) == api.SV_OK  # a batch without requests: nothing to do
    for bad in (dict(V=0), dict(ld=99), dict(ld=1 << 62), dict(R=-1), dict(dt=2), dict(T=0.0), dict(T=-1.0), dict(T=INF), dict(T=1e-31), dict(T=1e31),
                dict(T=math.nan), dict(n=-1), dict(n=33), dict(tok=None), dict(B=1), dict(B=2, cu=FAKE), dict(B=2, ln=FAKE),
                dict(B=-1, cu=FAKE, ln=FAKE), dict(z=None), dict(z=MISALIGNED), dict(tok=MISALIGNED), dict(lp=MISALIGNED),
                dict(rank=MISALIGNED), dict(ent=MISALIGNED), dict(ids=MISALIGNED), dict(tlp=MISALIGNED), dict(st=MISALIGNED)):
        assert _call(lib, **bad) == E, bad


def test_binding_refuses(lib):
    with pytest.raises(ValueError):
        api.sv_token_logprobs(torch.zeros(3, 8), torch.zeros(3, dtype=torch.int32))


# ---------------------------------------------------------------------------
# Against 64 bits
# ---------------------------------------------------------------------------
def _reference(z, tok, T, n):
    """(lp, rank, entropy, ids, top lp, E|t|) of the rows of z (CPU, any type) in 64 bits."""
    z = z.double()
    m = z.max(1, keepdim=True).values
    t = (z - m) / T
    lse = t.exp().sum(1, keepdim=True).log()
    lp = t - lse
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    spread = torch.where(p > 0, p * t.abs(), torch.zeros_like(p)).sum(1)
    value, ids = torch.sort(z + 0.0, dim=1, descending=True, stable=True)
    value, ids = value[:, :n], ids[:, :n]
    top = torch.where(value == -INF, torch.full_like(value, -INF), lp.gather(1, ids))
    ids = torch.where(value == -INF, torch.full_like(ids, -1), ids)
    if n > z.shape[1]:
        pad = (z.shape[0], n - z.shape[1])
        ids = torch.cat([ids, torch.full(pad, -1)], 1)
        top = torch.cat([top, torch.full(pad, -INF, dtype=torch.float64)], 1)
    zt = z.gather(1, tok.long()[:, None])
    rank = 1 + (z > zt).sum(1) + ((z == zt) & (torch.arange(z.shape[1])[None] < tok[:, None])).sum(1)
    return lp.gather(1, tok.long()[:, None])[:, 0], rank, ent, ids, top, spread


def _tolerances(V, spread):
    """Absolute error of ln S (eps) and of the entropy, worst case. Each term
    2^((z - m) c) has the rounding of the difference, of c and of the product
    (3 halves of eps of its exponent, so 1.5 * 2^-23 |t| relative in all) and
    2^-22 of the exponential; a thread adds at most V/256 + 8 of them one after
    another, half an eps each, and the rest is joined in double."""
    rel = 1.5 * 2.0 ** -23 * spread + 2.0 ** -22 + (V / 256 + 8) * 2.0 ** -24
    return rel, rel * (2 + 2 * spread)


def _check(z, tok, T, n, got, rows=None):
    lp, rank, ent, ids, top, spread = _reference(z, tok, T, n)
    eps, eps_h = _tolerances(z.shape[1], spread)
    if rows is None:
        rows = torch.arange(z.shape[0])
    close = lambda a, b, tol: bool(((a == b) | ((a - b).abs() <= tol + b.abs() * 2.0 ** -22)).all())  # noqa: E731
    g = [None if x is None else x.cpu()[rows] for x in got]
    assert torch.equal(g[1].long(), rank), (g[1], rank)
    assert torch.equal(g[3].long(), ids)
    assert close(g[0].double(), lp, eps), (g[0], lp)
    assert close(g[2].double(), ent, eps_h), (g[2], ent)
    assert close(g[4].double(), top, eps[:, None])


def _logits(R, V, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    z = torch.randn(R, V, generator=gen) * 2.5
    at = torch.randint(0, V, (R, 9), generator=gen)
    z.scatter_(1, at, 4 + 10 * torch.rand(R, 9, generator=gen))
    tok = torch.where(torch.arange(R) % 2 == 0, at[:, 4], torch.randint(0, V, (R,), generator=gen))
    return z.to(dtype), tok.to(torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,R,n,T", [(1, 3, 4, 1.0), (5, 7, 8, 0.5), (33, 40, 32, 1.3), (1000, 17, 20, 0.7), (4097, 9, 5, 1.0),
                                     (32000, 5, 5, 1.0), (32000, 1, 20, 1.0), (151936, 30, 20, 0.7), (256000, 3, 32, 2.0),
                                     (128255, 333, 1, 1.0), (32000, 700, 0, 1.0)])
def test_rows(cuda_lib, dtype, V, R, n, T):
    z, tok = _logits(R, V, dtype, 1000 + V + R)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.sv_token_logprobs(z.cuda(), tok.cuda(), temperature=T, n_top=max(n, 1), status=status)
    if n == 0:
        none = api.sv_token_logprobs(z.cuda(), tok.cuda(), temperature=T)
        assert none.top_ids is None and torch.equal(none.logprob, got.logprob) and torch.equal(none.rank, got.rank)
    _check(z, tok, T, max(n, 1), got)
    assert int(status) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,ld,first", [(1000, 1008, 0), (1000, 1001, 0), (1003, 1024, 1), (4096, 4104, 8), (40000, 40007, 3)])
def test_strides_and_alignment(cuda_lib, dtype, V, ld, first):
    R = 6
    z, tok = _logits(R, V, dtype, V + ld)
    buf = torch.full((R * ld + first,), float("nan"), dtype=dtype, device="cuda")  # what lies between the rows is not read
    view = buf[first:].view(-1)[: R * ld].view(R, ld)[:, :V]
    view.copy_(z)
    _check(z, tok, 0.9, 7, api.sv_token_logprobs(view, tok.cuda(), temperature=0.9, n_top=7))


def _shapes(V, dtype):
    """Rows whose order is hard: ties, masks, order, extremes."""
    asc = torch.arange(V, dtype=torch.float32) / V * 20
    rows = [torch.zeros(V), torch.full((V,), -3.0e38), asc, asc.flip(0), torch.full((V,), -INF), torch.full((V,), -INF)]
    rows[4][V // 2] = 1.5                                       # one token is allowed
    rows[5][torch.arange(0, V, max(1, V // 7))] = -2.0          # a few are, all alike
    saw = (torch.arange(V) % 97).float() / 8                    # long ties of the largest value
    zero = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)     # two zeros are one value
    low = torch.full((V,), torch.finfo(dtype).min)              # a mask of the type's lowest value
    low[V - 1] = 3.0
    low[0] = 3.0
    two = torch.full((V,), 1.0)
    two[V - 1] = 2.0
    block = torch.randn(V, generator=torch.Generator().manual_seed(5))
    block[: V // 2] = -INF                                      # half the vocabulary is masked
    far = torch.full((V,), -80.0)
    far[V // 3] = 90.0
    least = torch.full((V,), torch.finfo(dtype).min)            # nothing above the lowest value, and a padded tail
    least[V // 2:] = -INF
    huge = -1.0e6 - 8192.0 * (torch.arange(V) % 5)              # values whose next one is further off than any exponent reaches
    up = torch.full((V,), 2.0e38)
    up[V // 2:] = 1.0e38
    return torch.stack(rows + [saw, zero, low, two, block, far, least, huge, up]).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2, 64, 5000, 70001, 151936])
@pytest.mark.parametrize("copies", [1, 60])
def test_ties_masks_and_orders(cuda_lib, dtype, V, copies):
    z = _shapes(V, dtype).repeat(copies, 1) if V < 10000 or copies == 1 else _shapes(V, dtype).repeat(4, 1)
    tok = torch.tensor([V - 1, 0, V // 2, V // 3] * z.shape[0])[: z.shape[0]].to(torch.int32)
    got = api.sv_token_logprobs(z.cuda(), tok.cuda(), n_top=32)
    _check(z, tok, 1.0, 32, got)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1e-8, 1e-3, 50.0, 1e9])
def test_extreme_temperatures(cuda_lib, dtype, T):
    z, tok = _logits(5, 9000, dtype, 21)
    z[1, 100:8000] = -INF
    z[2, : 4000] = -INF
    tok[1], tok[2] = 3, 8999
    _check(z, tok, T, 9, api.sv_token_logprobs(z.cuda(), tok.cuda(), temperature=T, n_top=9))


@pytest.mark.gpu
@pytest.mark.parametrize("R", [4, 400])
def test_committed_rows_only(cuda_lib, R):
    """With a verify call's offsets and lengths: the other rows are neither read nor written, rows past the last request neither."""
    gen = torch.Generator().manual_seed(R)
    V, spare = 2000, 5
    K = torch.randint(0, 8, (R,), generator=gen)
    cu = torch.zeros(R + 1, dtype=torch.int32)
    cu[1:] = K.cumsum(0)
    n = (torch.rand(R, generator=gen) * (K + 2)).long().clamp(max=K + 1)  # zero among them
    rows = torch.cat([torch.arange(int(a), int(a) + int(m)) + b for b, (a, m) in enumerate(zip(cu[:-1], n))])
    total = int(cu[-1]) + R + spare
    z, tok = _logits(total, V, torch.bfloat16, R)
    masked = torch.full_like(z, float("nan"))
    masked[rows] = z[rows]
    tok_m = torch.full_like(tok, -1)
    tok_m[rows] = tok[rows]
    out = [torch.full((total,), 7.0, device="cuda"), torch.full((total,), 7, dtype=torch.int32, device="cuda"),
           torch.full((total,), 7.0, device="cuda"), torch.full((total, 3), 7, dtype=torch.int32, device="cuda"),
           torch.full((total, 3), 7.0, device="cuda")]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.sv_token_logprobs(masked.cuda(), tok_m.cuda(), cu_draft=cu.cuda(), out_len=n.to(torch.int32).cuda(), n_top=3,
                                out_logprob=out[0], out_rank=out[1], out_entropy=out[2], out_top_ids=out[3],
                                out_top_logprobs=out[4], status=status)
    _check(z[rows], tok[rows], 1.0, 3, got, rows)
    assert int(status) == 0
    rest = torch.ones(total, dtype=torch.bool)
    rest[rows] = False
    assert all(bool((x.cpu()[rest] == 7).all()) for x in out)


@pytest.mark.gpu
def test_data_errors(cuda_lib):
    V = 3001
    z, tok = _logits(6, V, torch.float32, 3)
    z[1] = -INF
    z[2, 17] = float("nan")
    z[3, 2999] = INF
    tok[4], tok[5] = V, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.sv_token_logprobs(z.cuda(), tok.cuda(), n_top=2, status=status)
    assert int(status) == api.SV_DATA_BAD_LOGIT | api.SV_DATA_EMPTY_ROW | api.SV_DATA_BAD_TOKEN
    lp, rank, ent, ids, top = (x.cpu() for x in got)
    assert lp[1:].isnan().all() and rank[1:].eq(0).all()
    assert ent[1:4].isnan().all() and ids[1:4].eq(-1).all() and top[1:4].isnan().all()
    ok = torch.tensor([0, 4, 5])
    want = _reference(z[ok], torch.zeros(3, dtype=torch.int32), 1.0, 2)
    assert torch.equal(ids[ok].long(), want[3]) and (top[ok] - want[4]).abs().max() < 1e-4 and (ent[ok] - want[2]).abs().max() < 1e-3
    # Offsets that decrease and lengths beyond the window: those rows stay as they were, the others are right.
    z, tok = _logits(8, V, torch.float32, 4)
    for cu, n, bad in (([0, 3, 2, 5], [1, 1, 1], True), ([0, 1, 3, 5], [3, 1, 1], True), ([0, 1, 3, 5], [-1, 1, 1], True),
                       ([1, 2, 3, 5], [1, 1, 1], True), ([0, 1, 3, 5], [2, 3, 3], False)):
        status.zero_()
        api.sv_token_logprobs(z.cuda(), tok.cuda(), cu_draft=torch.tensor(cu, dtype=torch.int32).cuda(),
                              out_len=torch.tensor(n, dtype=torch.int32).cuda(), status=status)
        assert (int(status) == api.SV_DATA_BAD_OFFSETS) == bad, cu


@pytest.mark.gpu
def test_streams_graphs_and_repeats(cuda_lib):
    """Two streams at once, a captured call replayed on new inputs, and the same bits every time."""
    z, tok = _logits(900, 32000, torch.bfloat16, 8)
    zc, tc = z.cuda(), tok.cuda()
    want = api.sv_token_logprobs(zc, tc, n_top=20)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [api.sv_token_logprobs(zc, tc, n_top=20, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    small, st = zc[:5].clone(), tc[:5].clone()
    api.sv_token_logprobs(small, st, n_top=20)
    graph = torch.cuda.CUDAGraph()
    src = zc[300:305].clone()
    with torch.cuda.graph(graph):
        small.copy_(src)  # a copy before the kernel, and one behind it
        out = api.sv_token_logprobs(small, st, n_top=20)
        after = out.logprob.clone()
    st.copy_(tc[300:305])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(after, out.logprob)
    torch.cuda.synchronize()
    _check(z[300:305], tok[300:305], 1.0, 20, out)


@pytest.mark.gpu
def test_of_a_verify_call(cuda_lib):
    """The committed tokens of spec_verify and their log probabilities: at temperature T, exp(logprob) of an accepted draft token is
    the p(x) that the verify call reports."""
    import parity
    from speculative_decoding_verification_27_gb300 import workloads as W
    b = W.config3(seed=77, B=24)
    db = parity.to_device(b)
    tokens, n, probs = api.spec_verify(db.target, db.draft, db.draft_tokens, db.cu_draft, db.uniforms, db.temperature, db.mode)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.sv_token_logprobs(db.target, tokens, cu_draft=db.cu_draft, out_len=n, temperature=db.temperature, n_top=4,
                                status=status)
    assert int(status) == 0
    seen = 0
    for i, m in enumerate(n.cpu().tolist()):
        r0 = int(db.cu_draft[i]) + i
        for j in range(m - 1):  # accepted slots
            p = float(probs[r0 + j, 0])
            assert abs(math.exp(float(got.logprob[r0 + j])) - p) <= 1e-5 * p + 1e-7
            seen += 1
    assert seen > 10


def _masked(V, dtype, value):
    """Rows of which all but a few tokens hold one large negative value; the allowed ones lie first, last, in the middle, anywhere."""
    gen = torch.Generator().manual_seed(V)
    z = torch.full((6, V), value)
    at = [range(4), range(V - 4, V), range(V // 2, V // 2 + 4), torch.randperm(V, generator=gen)[:40].tolist(),
          [V // 3, V // 2, V - 2, V - 1], list(range(0, V, max(1, V // 9)))]
    for r, x in enumerate(at):
        z[r, list(x)] = 3.0 * torch.randn(len(x), generator=gen)
    z[4, : V // 4] = -INF  # a mask of another kind beside it
    return z.to(dtype), torch.tensor([x[3] for x in at], dtype=torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,copies", [(5000, 1), (70001, 1), (151936, 1), (32000, 60)])
@pytest.mark.parametrize("value,T", [(torch.finfo(torch.bfloat16).min, 1.0), (torch.finfo(torch.float32).min / 2, 0.7), (-3.0e38, 1.0),
                                     (-1.0e38, 0.3), (-1.0e30, 1.0e-9), (-1.0e9, 1.0), (-1.0e4, 0.5)])
def test_masks_of_finite_values(cuda_lib, dtype, V, copies, value, T):
    """A masked token's term is nothing in the entropy, whatever finite value the mask has and whatever was seen before it."""
    z, tok = (x.repeat((copies,) + (1,) * (x.dim() - 1)) for x in _masked(V, dtype, value))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.sv_token_logprobs(z.cuda(), tok.cuda(), temperature=T, n_top=3, status=status)
    assert int(status) == 0
    _check(z, tok, T, 3, got)
    assert torch.equal(api.sv_token_logprobs(z.cuda(), tok.cuda(), temperature=T).entropy, got.entropy)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size,T", [(2.0 ** 60, 2.0 ** -100), (1.0e37, 1.0e-3), (1.0e30, 1.0e-20), (2.0 ** 90, 2.0 ** 80), (5.0e37, 2.0 ** 96)])
@pytest.mark.parametrize("V", [64, 9001, 128000])
def test_temperatures_beside_the_step_of_the_type(cuda_lib, dtype, size, T, V):
    """Logits whose neighbouring values lie further apart than any exponent reaches, and rows where they just do not."""
    gen = torch.Generator().manual_seed(V)
    z = (torch.randn(5, V, generator=gen) * size).to(dtype)
    z[1, : V // 2] = -INF
    z[2] = -z[2].float().abs().to(dtype)
    top = z.max(1, keepdim=True).values
    at = torch.stack([torch.randperm(V, generator=gen)[:3] for _ in range(5)])
    z.scatter_(1, at, top.expand(5, 3))  # three or four equal largest values
    z[3, at[3, 0]] = torch.nextafter(top[3], torch.full_like(top[3], -INF))[0]
    tok = at[:, 2].to(torch.int32)
    _check(z, tok, T, 2, api.sv_token_logprobs(z.cuda(), tok.cuda(), temperature=T, n_top=2))


def test_temperature_range(lib):
    """Above 2^96 what is zero beside a maximum near fp32's lowest value lies below that, and -inf could not be told from it."""
    assert _call(lib, T=2.0 ** 96, R=0) == _call(lib, T=2.0 ** -100, R=0) == api.SV_OK
    assert _call(lib, T=2.0 ** 96 * 1.001, R=0) == _call(lib, T=2.0 ** -101, R=0) == api.SV_ERR_INVALID_ARG
