"""Where the adapters' out may lie."""
import pytest
import torch

from tests.test_gpu_adapters import _adapters, _apply, _check, _make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("y", ["fp32", "bf16"])
def test_columns_of_one_buffer_are_taken(y):
    """x, base and out side by side in rows of one pitch share no byte."""
    K, N = 64, 40
    s = _make([3, 20, 1], [1, -1, 0], K, N, 16, 2, x=y, y=y, seed=6)
    buf = torch.full((s["T"], K + 2 * N + 24), 3.0, dtype=s["x"].dtype, device="cuda")
    for k, at, n in (("x", 0, K), ("base", K, N), ("out", K + N + 8, N)):
        view = buf[:, at:at + n]
        view.copy_(s[k])
        s[k] = view
    _apply(_adapters(s), s)
    _check(s, s["out"])
    assert (buf[:, K + N:K + N + 8] == 3.0).all() and (buf[:, K + 2 * N + 8:] == 3.0).all()


def test_an_out_over_x_or_beside_base_is_refused():
    """base is read ahead of what is written, and x by all blocks of a row while some write."""
    from speculative_decoding_verify_ragged_gb300 import SdvError
    s = _make([4, 8], [0, 1], 32, 32, 8, 2, x="fp32", y="fp32")
    ad = _adapters(s)
    buf = torch.randn((s["T"] + 2, 48), device="cuda")
    before = buf.clone()
    T = s["T"]
    for x, base, out in ((buf[:T, :32], s["base"], buf[:T, :32]), (buf[:T, :32], s["base"], buf[:T, 16:]), (s["x"], buf[:T, :32], buf[:T, 8:40]),
                         (s["x"], buf[:T, :32], buf[1:T + 1, :32]), (buf[:T, :32], buf[1:T + 1, :32], buf[1:T + 1, :32])):
        with pytest.raises(SdvError):
            ad.apply(x, base, out, s["row_offsets"], s["adapter_ids"], s["status"])
    torch.cuda.synchronize()
    assert torch.equal(buf, before) and s["status"].item() == 0
    _apply(ad, s)
    _check(s, s["out"])


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 40])
def test_buffers_of_the_most_rows(T):
    """A launch planned for as many rows as the count holds; only the requests' rows are touched (columns of one buffer, so that no
    rows are taken to overlap).  Items of 32 or 64 rows are counted past 32 bits on the way."""
    import ctypes
    from speculative_decoding_verify_ragged_gb300 import _abi
    s = _make([3, 20, 1], [1, 0, -1], 64, 40, 16, 2, x="fp32", y="fp32", seed=6)
    buf = torch.full((s["T"], 160), 3.0, device="cuda")
    for k, at, n in (("x", 0, 64), ("base", 64, 40), ("out", 112, 40)):
        view = buf[:, at:at + n]
        view.copy_(s[k])
        s[k] = view
    ad = _adapters(s, max_rows=T)
    r = _abi.SdvAdapterRows(3, T, s["row_offsets"].data_ptr(), s["adapter_ids"].data_ptr(), s["x"].data_ptr(), 1, 160, s["base"].data_ptr(),
                            s["out"].data_ptr(), 1, 160, 160)
    rc = ad.lib.sdv_adapters_apply(ad.handle, ctypes.byref(r), s["status"].data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    _check(s, s["out"])
