"""GPU tests of the numerics of the dense MLA attention where they can go wrong
quietly: many rescaled blocks, probabilities far below a row's largest, seen and
unseen infinities and NaN, far exponents.  The reference is the definition in 64
bits (dense_cases.reference, or written out here)."""
import math

import pytest
import torch

from dense_cases import BF16, FP8, Call, Latents
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
