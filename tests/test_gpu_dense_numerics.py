"""GPU tests of the numerics of the dense MLA attention where they can go wrong
quietly: many rescaled blocks, probabilities far below a row's largest, seen and
unseen infinities and NaN, far exponents.  The reference is the definition in 64
bits (dense_cases.reference, or written out here)."""
import math

import pytest
import torch

from dense_bounds import check_elements, check_rms, check_units, exact_rows, seen_of
from dense_cases import BF16, FP8, Call, Latents, check
from deepseek_sparse_attention_mqa_gb300 import _abi, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    _abi.lib()


# ------------------------------------------------ the any-shape kernel's factors

@pytest.mark.parametrize("fmt,heads,d_qk,d_v,page", [(BF16, 4, 80, 16, 64), (BF16, 16, 80, 64, 16), (FP8, 8, 128, 112, 32),
                                                     (FP8, 3, 576, 512, 16)])
@pytest.mark.parametrize("L", [64, 333, 640])
def test_maximum_grows_with_every_block(fmt, heads, d_qk, d_v, page, L):
    """Scores that grow from key to key, so that every block, the last one too, rescales
    what came before: the sums and the output's factors must not meet."""
    lat = Latents(fmt, d_qk, page, [L], seed=L)
    c = Call(lat, [L], [2], heads, d_v, seed=3, scale=1.0)
    # q along one dim whose key element grows by about 0.05 a key
    ramp = (0.05 * torch.arange(L, dtype=torch.float64, device="cuda")).float()
    k = lat.rows[0].float()
    k[:, d_qk - 1] = ramp
    _store(lat, 0, k)
    c.q.mul_(0.02)
    c.q[..., d_qk - 1] = 1.0
    ref = c.ref()
    first = None
    for _ in range(12):
        c.out.fill_(7)
        c.lse.fill_(7)
        c.run()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        # the output's half step of bf16, 2^-8 of itself; scores accumulated in fp32 (d_qk 2^-23 of
        # sum |q k|, in the probability and in its normaliser); P as two bf16, 2^-16; exp2 and sums 2^-20
        ds = lat.D * 2.0 ** -23 * float(torch.einsum("nhd,kd->nhk", c.q.double().abs(), lat.rows[0].abs()).max())
        tol = 2.0 ** -8 * ref[0].abs() + (2 * ds + 2.0 ** -16 + 2.0 ** -20) * _mag(c)
        assert bool(((c.out.double() - ref[0]).abs() <= tol).all())
        assert bool(((c.lse.double() - ref[1]).abs() <= ds + 2.0 ** -20 + 2.0 ** -22 * ref[1].abs()).all())
        if first is None:
            first = c.out.clone(), c.lse.clone()
        assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)


def _store(lat, b, rows):
    """Put fp32 rows into sequence b's pages, in the cache's format, and keep what the cache then holds."""
    L, D, page = rows.shape[0], lat.D, lat.page
    if lat.fmt == FP8:
        s = rows.abs().amax(-1, keepdim=True).clamp_min(1e-30) / 448
        c = (rows / s).to(torch.float8_e4m3fn)
        lat.codes[b], lat.scale_rows[b] = c.double(), s[:, 0].double()
        lat.rows[b] = c.double() * s.double()
    else:
        c = rows.to(torch.bfloat16)
        lat.codes[b] = lat.rows[b] = c.double()
    raw = c.view(torch.uint8)
    for j in range(-(-L // page)):
        p, n = int(lat.table[b, j]), min(page, L - j * page)
        lat.values[p, :page * lat.tok].view(page, lat.tok)[:n, :raw.shape[1]] = raw[j * page:j * page + n]
        if lat.fmt == FP8:
            lat.scales[p, :n] = s[j * page:j * page + n, 0]


def _mag(c):
    """sum_j p_j |v_j| of every output of a one-sequence call, in 64 bits."""
    k = c.lat.rows[0]
    L, n = k.shape[0], c.rows
    s = c.scale * torch.einsum("nhd,kd->nhk", c.q[:n].double(), k)
    seen = torch.arange(L, device=k.device)[None, :] <= (L - n + torch.arange(n, device=k.device))[:, None]
    p = torch.softmax(s.masked_fill(~seen[:, None, :], -math.inf), -1)
    return torch.einsum("nhk,kv->nhv", p, k[:, :c.d_v].abs())


# ------------------------------------- probabilities far below the row's largest

def _call(lat, L, news, heads, d_v=512, q=None, scale=1.0, seed=4):
    c = Call(lat, [L], [news], heads, d_v, seed=seed, scale=scale)
    if q is not None:
        c.q.copy_(q.expand_as(c.q))
    return c


def _checked(c, elements=True, rows=None):
    c.run()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    rows = rows or [0, c.rows // 2, c.rows - 1]
    ref, z, mag, noise, ds = exact_rows(c, rows)
    check_rms(c.out[rows], ref)
    if elements:
        check_elements(c.out[rows], c.lse[rows], ref, z, mag, noise, ds)


@pytest.mark.parametrize("L,news", [(16384, 160), (131072, 80)])
@pytest.mark.parametrize("above,sd", [(10.0, 0.01), (12.0, 0.3), (12.5, 0.5), (13.0, 1.0), (14.0, 0.3)])
@pytest.mark.parametrize("ratio", [1.0, 7.0])
def test_one_heavy_key_above_a_flat_context(L, news, above, sd, ratio):
    """A key (an attention sink) `above` nats over a long context whose values share a mean: each
    of the others is 2^-14 to 2^-20 of it and together they weigh as much.  `ratio`: their token
    scale over the heavy key's."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    lat = Latents(FP8, 576, 64, [L], seed=1)
    k = 0.5 + torch.randn((L, 576), generator=g, device="cuda")
    k[:, 575] = sd * torch.randn(L, generator=g, device="cuda")      # the score
    k[:, 574] = 16.0 * ratio                                          # the token scale
    k[9, 574], k[9, 575] = 16.0, above
    _store(lat, 0, k)
    q = 0.004 * torch.randn((1, 128, 576), generator=g, device="cuda")
    q[..., 574], q[..., 575] = 0.0, 1.0
    _checked(_call(lat, L, news, 128, q=q.to(torch.bfloat16)))


@pytest.mark.parametrize("spread,shift,qscale", [(0.3, 0.0, 1.0), (0.3, 0.5, 1.0), (0.3, 0.5, 0.6), (0.0, 0.5, 1.7)])
def test_scores_of_many_magnitudes(spread, shift, qscale):
    """Random latents whose magnitudes vary: the largest of 70000 scores lies far above what most of
    the softmax's mass does, in nats, and blocks' maxima differ by as much."""
    lat = Latents(FP8, 576, 64, [70000], seed=2, spread=spread)
    if shift:
        _store(lat, 0, (lat.rows[0] + shift).float())
    c = _call(lat, 70000, 80, 128, scale=1.0 / math.sqrt(192))
    c.q.mul_(qscale)
    _checked(c)


@pytest.mark.parametrize("heads", [128, 16])
def test_a_heavy_key_in_every_block(heads):
    """One key of every 128 heavy by 10 nats, the first by 6 more."""
    L = 32768
    lat = Latents(FP8, 576, 64, [L], seed=1)
    k = 0.5 + torch.randn((L, 576), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    k[:, 575] = 0.0
    k[:, 574] = 20.0
    k[::128, 575] = 10.0
    k[0, 575] = 16.0
    _store(lat, 0, k)
    q = torch.zeros((1, heads, 576), device="cuda")
    q[..., 575] = 1.0
    _checked(_call(lat, L, 160, heads, q=q.to(torch.bfloat16)))


def test_a_sink_and_then_rising_and_falling_contexts():
    """The block maxima fall by 25 nats, come back by 20 and fall again."""
    L = 65536
    lat = Latents(FP8, 576, 64, [L], seed=1)
    k = 0.5 + torch.randn((L, 576), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    lvl = torch.zeros(L, device="cuda")
    lvl[16384:32768] = 20.0
    lvl[32768:49152] = 8.0
    k[:, 575] = lvl + 0.3 * torch.randn(L, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    k[:, 574] = 30.0
    k[0, 575] = 25.0
    _store(lat, 0, k)
    q = torch.zeros((1, 128, 576), device="cuda")
    q[..., 575] = 1.0
    _checked(_call(lat, L, 80, 128, q=q.to(torch.bfloat16)))


# ------------------------------------------------------------- seen infinities

def _definition(c, window=None, sinks=0):
    """out and lse of every row from the definition in 64 bits, infinities included: a key
    with probability 0 still multiplies its value."""
    k = c.lat.rows[0]
    outs, lses = [], []
    L, n = c.lens[0], c.rows
    for i in range(n):
        vis = min(max(L - n + i + 1, 0), L)
        pos = torch.arange(vis, device=k.device)
        keep = (pos >= vis - window) | (pos < sinks) if window is not None else torch.ones_like(pos, dtype=torch.bool)
        x = k[pos[keep]]
        s = c.scale * (c.q[i].double()[:, None, :] * x[None]).sum(-1)
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - z[:, None])
        outs.append((p[:, :, None] * x[None, :, :c.d_v]).sum(1))
        lses.append(z)
    return torch.stack(outs), torch.stack(lses)


@pytest.mark.parametrize("heads,d_qk,d_v,page", [(16, 576, 512, 64), (128, 512, 512, 32), (4, 80, 64, 64), (16, 576, 512, 16),
                                                 (3, 576, 512, 64)])
@pytest.mark.parametrize("window", [None, 40])
@pytest.mark.parametrize("where", [250, 120, 299])
def test_seen_infinities_give_what_the_definition_gives(heads, d_qk, d_v, page, window, where):
    """A bf16 latent with an infinity: where its score is -inf its probability is 0, and 0 x inf is NaN
    in that element, whatever else the row's tile sees; where it is +inf or NaN the whole row is."""
    lat = Latents(BF16, d_qk, page, [300], seed=3)
    c = Call(lat, [300], [100], heads, d_v, seed=4)
    bad = {where: (5, float("inf")), where - 3: (11, -float("inf")), 7: (d_qk - 1, float("inf"))}
    c.q[..., 5] = -c.q[..., 5].abs() - 0.5                  # x inf: -inf
    c.q[..., 11] = c.q[..., 11].abs() + 0.5
    c.q[..., d_qk - 1] = -c.q[..., d_qk - 1].abs() - 0.5
    c.q[50, 0, 5] = 1.0                                     # one row sees +inf
    for p, (d, v) in bad.items():
        lat.rows[0][p, d] = v
        row = lat.values[int(lat.table[0, p // page]), (p % page) * lat.tok:(p % page + 1) * lat.tok]
        row[:2 * d_qk].view(torch.bfloat16)[d] = v
    c.run(window, 2)
    torch.cuda.synchronize()
    ref, z = _definition(c, window, 2)
    assert torch.equal(torch.isnan(c.out), torch.isnan(ref.to(torch.bfloat16)))
    fin = torch.isfinite(z)
    assert torch.equal(torch.isfinite(c.lse), fin)
    ok = ~torch.isnan(ref)
    # |out| < 8 here: 2^-8 of itself, and of the values' sum, as everywhere
    assert bool(((c.out.double() - ref)[ok].abs() <= 2.0 ** -8 * ref[ok].abs() + 0.03).all())
    assert bool(((c.lse.double() - z)[fin].abs() <= 1e-3).all())


@pytest.mark.parametrize("heads,d_qk,d_v,page", [(16, 576, 512, 64), (4, 80, 64, 64), (128, 576, 512, 64)])
@pytest.mark.parametrize("scale", [float("inf"), float("nan"), -float("inf")])
@pytest.mark.parametrize("window", [None, 40])
def test_token_scales_that_are_not_finite(heads, d_qk, d_v, page, scale, window):
    """An infinite or NaN token scale spoils the rows that see the token, whatever its score's sign, and
    no others."""
    lat = Latents(FP8, d_qk, page, [300], seed=3)
    c = Call(lat, [300], [100], heads, d_v, seed=4)
    bad = 250
    lat.scales[int(lat.table[0, bad // page]), bad % page] = scale
    c.run(window, 2)
    torch.cuda.synchronize()
    saw = torch.zeros(100, dtype=torch.bool, device="cuda")
    saw[50:(50 + window) if window else None] = True
    assert bool(torch.isnan(c.out[saw]).all())
    ref = c.ref(window, 2)
    check(c.out[~saw], c.lse[~saw], tuple(x[~saw] for x in ref))


# ------------------------------------------------------ NaN scales and queries

SMALL = [(BF16, 4, 80, 64, 64), (FP8, 4, 80, 64, 64), (BF16, 16, 576, 512, 64), (FP8, 16, 576, 512, 64), (FP8, 128, 512, 512, 32)]


@pytest.mark.parametrize("fmt,heads,d_qk,d_v,page", SMALL)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_queries_that_are_not_finite_in_rows_without_keys(fmt, heads, d_qk, d_v, page, value):
    """A row that sees nothing gives 0 and -inf whatever its q holds, beside rows that see keys; also
    where its keys' pages do not exist."""
    lat = Latents(fmt, d_qk, page, [3, 200], seed=3)
    lat.bt[1, :] = -1
    c = Call(lat, [3, 200], [5, 1], heads, d_v, seed=4)
    c.q[:2] = value
    c.q[5, :, 3] = value
    ref = c.ref()
    c.run()
    torch.cuda.synchronize()
    assert _abi.device_status(c.status) == _abi.DEV_BAD_INDEX
    for r in (0, 1, 5):
        assert bool((c.out[r] == 0).all()) and bool((c.lse[r] == float("-inf")).all())
    check(c.out[2:5], c.lse[2:5], tuple(x[2:5] for x in ref))


@pytest.mark.parametrize("fmt,heads,d_qk,d_v,page", SMALL)
def test_nan_softmax_scale(fmt, heads, d_qk, d_v, page):
    """NaN for every row that sees a key, 0 and -inf for those that see none."""
    lat = Latents(fmt, d_qk, page, [3], seed=3)
    c = Call(lat, [3], [5], heads, d_v, seed=4, scale=float("nan"))
    c.run()
    torch.cuda.synchronize()
    assert bool((c.out[:2] == 0).all()) and bool((c.lse[:2] == float("-inf")).all())
    assert bool(torch.isnan(c.out[2:]).all()) and bool(torch.isnan(c.lse[2:]).all())


@pytest.mark.parametrize("fmt,heads,d_qk,d_v,page", SMALL)
@pytest.mark.parametrize("power", [100, 107, 108, 109, 112, 124])
def test_queries_near_the_largest_bf16(fmt, heads, d_qk, d_v, page, power):
    """Rows of q around 2^power, with a softmax_scale that brings their scores back.  (At 2^124 only
    where q is scaled before it is multiplied; elsewhere the fp32 sums leave their range.)"""
    if power == 124 and (fmt, d_v) != (FP8, 512):
        return
    lat = Latents(fmt, d_qk, page, [200, 90], seed=3, spread=0.0)
    c = Call(lat, [200, 90], [3, 1], heads, d_v, seed=4, scale=2.0 ** -power / 14)
    c.q.copy_((c.q.float().clamp(-4, 4) * 2.0 ** power).to(torch.bfloat16))
    c.run()
    torch.cuda.synchronize()
    check(c.out, c.lse, c.ref())


# ---------------------------------------------- strides past what a tensor map holds

@pytest.mark.parametrize("fmt", [FP8, BF16])
def test_page_stride_past_two_to_the_40(fmt):
    """A cache of one page may state any page stride."""
    lat = Latents(fmt, 576, 64, [60], seed=3)
    c = Call(lat, [60], [2], 16, 512, seed=4)
    page = int(lat.table[0, 0])
    v = lat.values[page].clone()
    s = lat.scales[page].clone() if fmt == FP8 else None
    bt = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    c.cache = _abi.make_cache(fmt, 576, 64, 1, v, 1 << 41, lat.tok, s, 256 if fmt == FP8 else 0, 4 if fmt == FP8 else 0, bt)
    c.run()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    check(c.out, c.lse, c.ref())


@pytest.mark.parametrize("heads,d_qk,d_v,page", [(16, 576, 512, 64), (128, 512, 512, 32), (4, 80, 64, 64)])
@pytest.mark.parametrize("power", [-58, -40, 40, 59, 62, 70, 100])
def test_token_scales_of_far_powers(heads, d_qk, d_v, page, power):
    """All token scales times 2^power, the scores brought back by the softmax_scale."""
    lat = Latents(FP8, d_qk, page, [300, 90], seed=3)
    lat.scales.mul_(2.0 ** power)
    for b in range(2):
        lat.scale_rows[b] *= 2.0 ** power
        lat.rows[b] *= 2.0 ** power
    c = Call(lat, [300, 90], [3, 1], heads, d_v, seed=4, scale=2.0 ** -power / 14)
    c.run()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    check(c.out, c.lse, c.ref())


# ------------------------------------------------------------ long and cut contexts

@pytest.mark.parametrize("fmt,heads,d_qk,d_v,page", [(FP8, 128, 576, 512, 64), (FP8, 16, 512, 512, 32), (BF16, 32, 576, 512, 64),
                                                     (BF16, 64, 80, 64, 64), (FP8, 16, 576, 512, 16)])
@pytest.mark.parametrize("lens,news,window", [([20000], [1], None), ([9001, 40, 15000, 0, 777], [1, 2, 3, 0, 1], None),
                                              ([15000, 7000], [1, 2], 6000)])
def test_cut_contexts_lose_and_repeat_no_block(fmt, heads, d_qk, d_v, page, lens, news, window):
    """Row by row against the bound that one missing or repeated block of keys exceeds."""
    lat = Latents(fmt, d_qk, page, lens, seed=heads)
    c = Call(lat, lens, news, heads, d_v, seed=heads + 1)
    c.run(window, 100)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    row = 0
    for b, n in enumerate(news):
        for i in range(n):
            p, v, ref = seen_of(c, b, i, window, 100)
            check_rms(c.out[row], ref)
            assert check_units(c.out[row], ref, p, v) > 0
            row += 1


@pytest.mark.parametrize("heads,d_qk,d_v,page", [(16, 576, 512, 64), (128, 512, 512, 32), (4, 80, 64, 64)])
@pytest.mark.parametrize("kind", ["negative", "zero", "mixed"])
def test_token_scales_of_either_sign_and_zero(heads, d_qk, d_v, page, kind):
    """Scales below zero flip their token, zeros among others give a key with score 0 and no value."""
    lat = Latents(FP8, d_qk, page, [900, 90], seed=3)
    for b, L in enumerate((900, 90)):
        f = torch.ones(L, dtype=torch.float64, device="cuda")
        if kind != "zero":
            f[::3] = -1.0
        if kind != "negative":
            f[1::5] = 0.0
        for j in range(-(-L // page)):
            n = min(page, L - j * page)
            lat.scales[int(lat.table[b, j]), :n] *= f[j * page:j * page + n].float()
        lat.scale_rows[b] *= f
        lat.rows[b] *= f[:, None]
    c = Call(lat, [900, 90], [5, 90], heads, d_v, seed=4)
    c.run()
    torch.cuda.synchronize()
    check(c.out, c.lse, c.ref())
    c.run(64, 3)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    check(c.out, c.lse, c.ref(64, 3))


def test_falling_references_and_cut_pieces_in_a_graph():
    """A captured call over a context with an early heavy key, replayed: the same bits as the first call."""
    L = 40000
    lat = Latents(FP8, 576, 64, [L], seed=1)
    k = 0.5 + torch.randn((L, 576), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    k[:, 575] = 0.0
    k[:, 574] = 16.0
    k[3, 575] = 12.0
    _store(lat, 0, k)
    q = torch.zeros((1, 128, 576), device="cuda")
    q[..., 575] = 1.0
    c = _call(lat, L, 20, 128, q=q.to(torch.bfloat16))
    _checked(c)
    out, lse = c.out.clone(), c.lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for _ in range(2):
        c.out.fill_(7)
        c.ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.out) and torch.equal(lse, c.lse)
