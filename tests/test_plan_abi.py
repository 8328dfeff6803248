"""Refusals of a plan whose outputs have room for more requests than the step, without a device."""
import ctypes


def test_room_for_fewer_requests_than_the_step_is_refused():
    from speculative_decoding_verify_ragged_gb300 import _abi
    lib = _abi.load_library()
    good = dict(B=2, T=8, new_rows=4096, lens=4096, page_table=4096, max_pages_per_seq=4, page_counts=4096, free_pages=4096,
                num_pool_pages=9, num_free=4096, row_offsets=4096)
    for max_b, want in ((-1, _abi.SDV_ERR_INVALID_ARG), (1, _abi.SDV_ERR_INVALID_ARG), (1025, _abi.SDV_ERR_CAPACITY)):
        t = _abi.SdvCacheTables(max_B=max_b, **good)
        assert lib.sdv_cache_plan(ctypes.byref(t), ctypes.c_void_p(4096), None) == want
    assert ctypes.sizeof(_abi.SdvCacheTables) == 14 * 8 + 8
