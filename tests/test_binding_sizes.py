"""Sizes past 32 bits in the bindings of adapters and sampling: never wrapped on their way into the C structs."""
import ctypes
import types

import pytest
import torch

STREAM = types.SimpleNamespace(cuda_stream=0)


def test_rows_of_the_adapters_are_not_wrapped():
    """The library is a recorder here."""
    from speculative_decoding_verify_ragged_gb300 import adapter
    from speculative_decoding_verify_ragged_gb300._abi import SdvAdapterRows
    seen = []
    ad = adapter.Adapters.__new__(adapter.Adapters)
    ad.lib = types.SimpleNamespace(sdv_adapters_apply=lambda h, r, status, raw: seen.append(ctypes.cast(r, ctypes.POINTER(SdvAdapterRows)).contents.T) or 0,
                                   sdv_adapters_destroy=lambda h: None)
    ad.handle, ad._index, ad.device, ad.k, ad.n = 1, -1, torch.device("cpu"), 8, 16
    i32 = dict(dtype=torch.int32)
    for rows in (4, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 4):
        x, y = torch.zeros((1, 8)).expand(rows, 8), torch.zeros((1, 16)).expand(rows, 16)
        call = lambda: ad.apply(x, y, y, torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32), stream=STREAM)  # noqa: E731
        if rows < 2 ** 31:
            call()
            assert seen[-1] == rows
        else:
            with pytest.raises(ValueError, match="2\\^31"):
                call()
    assert len(seen) == 2


@pytest.mark.gpu
def test_a_vocabulary_past_32_bits_is_refused():
    """2^32 + 100 columns are not 100."""
    from speculative_decoding_verify_ragged_gb300.sample import sample
    z = torch.empty((1, 2 ** 32 + 100), dtype=torch.bfloat16, device="cuda")
    tokens, status = torch.full((1,), -7, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        sample(z, status, uniforms=torch.zeros(1, device="cuda"), tokens=tokens)
    assert tokens.item() == -7 and status.item() == 0
