"""GPU tests of dsa_kv_gather_dequantize at the ends of its ranges of sizes."""
import pytest
import torch

from deepseek_sparse_attention_mqa_gb300 import _abi, build
from test_gpu_gather import BF16, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    _abi.lib()


def test_as_many_output_rows_as_an_integer_holds():
    """2^31 - 1 rows of 8 bf16 (34 GB), of which the ranges at either end are written."""
    rows = 2 ** 31 - 1
    cache, v, _, bt, tok, _ = make(BF16, 8, 4, 7, 2, 5, 3)
    cum = torch.tensor([0, 3, 3], dtype=torch.int32, device="cuda")
    out = torch.empty((rows, 8), dtype=torch.bfloat16, device="cuda")
    out[:8] = 9
    out[-24:] = 9
    _abi.kv_gather_dequantize(cache, cum, None, out)
    torch.cuda.synchronize()
    page = v[int(bt[0, 0])].view(torch.bfloat16).view(4, 8)
    assert torch.equal(out[:3], page[:3]) and bool((out[3:8] == 9).all()) and bool((out[-24:] == 9).all())
    cum = torch.tensor([rows - 20, rows - 20, rows], dtype=torch.int32, device="cuda")
    _abi.kv_gather_dequantize(cache, cum, None, out)
    torch.cuda.synchronize()
    want = torch.cat([v[int(p)].view(torch.bfloat16).view(4, 8) for p in bt[1]])
    assert torch.equal(out[-20:], want) and bool((out[-24:-20] == 9).all())
