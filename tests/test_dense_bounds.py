"""CPU checks of the bounds that long contexts are held to: a result that lacks a block of keys,
or holds one twice, is rejected wherever the block lies."""
import pytest
import torch

from dense_bounds import check_elements, check_rms, check_units, exact_rows, seen_of
from dense_cases import BF16, FP8, Call, Latents
from deepseek_sparse_attention_mqa_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("fmt,heads,d_qk,d_v", [(FP8, 16, 576, 512), (BF16, 16, 576, 512), (BF16, 64, 80, 64)])
def test_a_missing_or_repeated_unit_is_rejected(fmt, heads, d_qk, d_v):
    L = 8000
    lat = Latents(fmt, d_qk, 64, [L], seed=16, dev="cpu")
    c = Call(lat, [L], [1], heads, d_v, seed=17)
    ref, z, mag, noise, ds = exact_rows(c, [0])
    once = ref.to(torch.bfloat16)
    check_rms(once, ref)
    check_elements(once, z.float(), ref, z, mag, noise, ds)
    p, v, r = seen_of(c, 0, 0)
    assert check_units(once[0], r, p, v) >= 0.9 * (L // 32)
    for at, n in ((0, 128), (32, 32), (4096, 128), (4000, 32), (L - 64, 64), (L - 32, 32)):
        part = p[:, at:at + n]
        for sign in (-1.0, 1.0):                                  # without the keys, with them twice
            got = (r + sign * part @ v[at:at + n]) / (1 + sign * part.sum(-1, keepdim=True))
            with pytest.raises(AssertionError):
                check_units(got.to(torch.bfloat16), r, p, v)
