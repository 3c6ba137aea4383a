"""CPU checks: what the binding of the dense MLA attention and of the cache read-back refuses
before any call, because the kernels would read past a tensor's end."""
import pytest
import torch

from deepseek_sparse_attention_mqa_gb300 import _abi, build
from test_dense_refusals import cache


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    _abi.lib()


def tensors(rows=2):
    q = torch.zeros((rows, 16, 576), dtype=torch.bfloat16)
    return q, torch.zeros((rows, 16, 512), dtype=torch.bfloat16), torch.zeros((rows, 16))


def i32(n):
    return torch.zeros((n,), dtype=torch.int32)


@pytest.mark.parametrize("window", [False, True])
@pytest.mark.parametrize("lens,cum,batch", [(2, 2, None), (2, None, 3), (2, 3, 3), (3, 4, 4), (2, 1, 1)])
def test_attention_wants_a_length_and_rows_for_every_sequence(window, lens, cum, batch):
    """lens, cum: lengths of seq_lens and cum_q."""
    q, out, lse = tensors()
    kw = dict(cum_q=None if cum is None else i32(cum), batch=batch, stream=0)
    with pytest.raises(ValueError):
        if window:
            _abi.mla_attention_window(q, 0.1, cache(), i32(lens), 4, 0, out, lse, 512, **kw)
        else:
            _abi.mla_attention(q, 0.1, cache(), i32(lens), out, lse, 512, **kw)


def test_attention_wants_an_int32_status():
    q, out, lse = tensors()
    for bad in (torch.zeros((1,), dtype=torch.int64), torch.zeros((0,), dtype=torch.int32)):
        with pytest.raises((TypeError, ValueError)):
            _abi.mla_attention(q, 0.1, cache(), i32(2), out, lse, 512, status=bad, stream=0)
        with pytest.raises((TypeError, ValueError)):
            _abi.kv_gather_dequantize(cache(), i32(3), None, torch.zeros((4, 576)), status=bad, stream=0)


@pytest.mark.parametrize("cum,starts,batch", [(3, 1, None), (3, None, 3), (4, 2, 3), (0, None, None)])
def test_gather_wants_rows_and_a_start_for_every_sequence(cum, starts, batch):
    with pytest.raises(ValueError):
        _abi.kv_gather_dequantize(cache(), i32(cum), None if starts is None else i32(starts), torch.zeros((4, 576)),
                                  batch=batch, stream=0)


def test_longer_tensors_than_the_batch_are_taken():
    """A padded batch: the first `batch` sequences of longer tensors (the call gets as far as the library, which
    wants a workspace)."""
    q, out, lse = tensors()
    with pytest.raises(_abi.DSAError) as e:
        _abi.mla_attention(q, 0.1, cache(), i32(8), out, lse, 512, cum_q=i32(9), batch=2, stream=0)
    assert e.value.status == _abi.DSA_ERR_INVALID_ARG


def test_the_block_table_has_a_row_for_every_sequence():
    q, out, lse = tensors()
    v, sc, bt = torch.zeros((4, 64 * 576), dtype=torch.uint8), torch.zeros((4, 64)), torch.zeros((1, 3), dtype=torch.int32)
    c = _abi.make_cache(_abi.FMT_FP8, 576, 64, 4, v, 64 * 576, 576, sc, 256, 4, bt)
    with pytest.raises(ValueError):
        _abi.mla_attention(q, 0.1, c, i32(2), out, lse, 512, stream=0)
    with pytest.raises(ValueError):
        _abi.mla_attention_window(q, 0.1, c, i32(2), 4, 0, out, lse, 512, stream=0)
    with pytest.raises(ValueError):
        _abi.kv_gather_dequantize(c, i32(3), None, torch.zeros((4, 576)), stream=0)
