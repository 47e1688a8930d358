"""What the norm, gate, combination and NVFP4 matrix-vector calls refuse, on
the host: status codes of the C ABI (the pointers are never read: validation
fails first) and the Python entry points' ValueErrors."""
import ctypes

import pytest
import torch

import mxfp8_block_scaled_warp_b200 as f
from mxfp8_block_scaled_warp_b200 import moe

INVALID, ALIGNMENT, UNSUPPORTED, WORKSPACE = 1, 2, 3, 7
P = 1 << 20                               # an aligned address
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from mxfp8_block_scaled_warp_b200 import build
    build.build()
    return f.load()


def _refused(call, good, cases):
    """Every case replaces arguments of the good call by position."""
    for changes, status in cases:
        args = list(good)
        for i, v in changes.items():
            args[i] = v
        assert call(*args) == status, (changes, status)


def test_rmsnorm(lib):
    # fmt x ld res w rows cols eps h y q scales rstd stream
    good = [f.MXFP8, P, 256, P, P, 4, 256, 1e-6, P, P, P, P, P, None]
    _refused(lib.fpq_rmsnorm_quantize, good, [
        ({5: -1}, INVALID), ({5: 1 << 31}, INVALID), ({6: 0}, INVALID), ({6: 252}, INVALID), ({6: 264}, INVALID),
        ({2: 248}, INVALID), ({2: 260}, INVALID), ({6: 32776, 2: 32776}, INVALID), ({6: 248}, INVALID),
        ({0: f.FP8_1x128, 6: 192}, INVALID), ({0: f.NVFP4}, UNSUPPORTED), ({0: f.FP8_128x128}, UNSUPPORTED),
        ({0: 9}, INVALID), ({7: NAN}, INVALID), ({7: -1.0}, INVALID), ({7: INF}, INVALID),
        ({10: None}, INVALID), ({11: None}, INVALID), ({9: None, 10: None, 11: None}, INVALID),
        ({1: None}, INVALID), ({4: None}, INVALID), ({1: P + 2}, ALIGNMENT), ({3: P + 8}, ALIGNMENT),
        ({8: P + 4}, ALIGNMENT), ({9: P + 4}, ALIGNMENT), ({10: P + 8}, ALIGNMENT), ({11: P + 1}, ALIGNMENT),
        ({12: P + 4}, ALIGNMENT)])
    assert lib.fpq_rmsnorm_quantize(*(good[:5] + [0] + good[6:])) == 0          # no rows: nothing to do


def test_rmsnorm_backward(lib):
    # dy x ld w rstd dres rows cols dx dweight ws wsb stream
    good = [P, P, 256, P, P, P, 4, 256, P, P, P, 1 << 30, None]
    _refused(lib.fpq_rmsnorm_backward, good, [
        ({6: -1}, INVALID), ({7: 12, 2: 16}, INVALID), ({2: 128}, INVALID), ({7: 40000, 2: 40000}, INVALID),
        ({0: None}, INVALID), ({4: None}, INVALID), ({8: None}, INVALID), ({5: P + 2}, ALIGNMENT),
        ({9: P + 4}, ALIGNMENT)])
    assert lib.fpq_rmsnorm_backward_workspace_bytes(4, 12) == 0


def test_gate(lib):
    # logits dtype bias tokens E score n_group topk_group group_top topk renorm scale ids weights stream
    good = [P, 1, P, 16, 64, 1, 8, 4, 2, 8, 1, 1.0, P, P, None]
    _refused(lib.fpq_moe_gate, good, [
        ({1: 2}, INVALID), ({3: -1}, INVALID), ({4: 0}, INVALID), ({4: 1025}, INVALID), ({5: 2}, INVALID),
        ({6: 0}, INVALID), ({6: 7}, INVALID), ({6: 64}, INVALID), ({7: 0}, INVALID), ({7: 9}, INVALID),
        ({8: 0}, INVALID), ({8: 3}, INVALID), ({9: 0}, INVALID), ({9: 33}, INVALID), ({6: 32, 7: 3}, INVALID),
        ({4: 8, 6: 8, 9: 2}, INVALID), ({4: 4, 6: 1, 7: 1, 9: 5}, INVALID), ({3: 1 << 30}, INVALID),
        ({10: 2}, INVALID), ({0: None}, INVALID), ({12: None}, INVALID), ({13: None}, INVALID),
        ({0: P + 4}, ALIGNMENT), ({2: P + 4}, ALIGNMENT)])
    assert lib.fpq_moe_gate(*(good[:3] + [0] + good[4:])) == 0
    # logits dtype ids dweights tokens E score topk renorm scale dlogits stream
    good = [P, 0, P, P, 16, 64, 0, 8, 1, 1.0, P, None]
    _refused(lib.fpq_moe_gate_backward, good, [
        ({1: -1}, INVALID), ({4: -1}, INVALID), ({5: 2000}, INVALID), ({6: 3}, INVALID), ({7: 0}, INVALID),
        ({7: 40}, INVALID), ({8: -1}, INVALID), ({2: None}, INVALID), ({10: P + 2}, ALIGNMENT)])


def test_combine_and_rows(lib):
    # y dtype y_rows rows weights tokens topk hidden add out out_dtype stream
    good = [P, 0, 128, P, P, 16, 8, 64, P, P, 0, None]
    _refused(lib.fpq_moe_combine, good, [
        ({1: 3}, INVALID), ({2: -1}, INVALID), ({2: 1 << 31}, INVALID), ({5: -1}, INVALID), ({6: 0}, INVALID),
        ({6: 33}, INVALID), ({7: 60}, INVALID), ({7: 0}, INVALID), ({10: 2}, INVALID), ({3: None, 2: 127}, INVALID),
        ({5: 1 << 28}, INVALID), ({0: None}, INVALID), ({4: None}, INVALID), ({9: None}, INVALID),
        ({3: P + 4}, ALIGNMENT), ({8: P + 2}, ALIGNMENT), ({0: P + 8}, ALIGNMENT)])
    # dout dtype y dtype y_rows rows weights tokens topk hidden dy dweights stream
    good = [P, 1, P, 0, 128, P, P, 16, 8, 64, P, P, None]
    _refused(lib.fpq_moe_combine_backward, good, [
        ({1: 5}, INVALID), ({9: 4}, INVALID), ({5: None, 4: 100}, INVALID), ({0: None}, INVALID), ({10: None}, INVALID),
        ({11: None}, INVALID), ({5: P + 4}, ALIGNMENT), ({10: P + 8}, ALIGNMENT)])
    # ids tokens topk E ws wsb dst_row0 rows stream
    good = [P, 16, 8, 64, P, 1 << 30, P, P, None]
    _refused(lib.fpq_moe_pair_rows, good, [
        ({1: -1}, INVALID), ({2: 40}, INVALID), ({3: 0}, INVALID), ({0: None}, INVALID), ({7: P + 4}, ALIGNMENT),
        ({4: None}, WORKSPACE), ({5: 8}, WORKSPACE)])


def test_gemv(lib):
    # x m wq ws wg n k y dtype stream
    good = [P, 4, P, P, P, 64, 256, P, 0, None]
    _refused(lib.fpq_gemv_nvfp4, good, [
        ({1: -1}, INVALID), ({1: 17}, INVALID), ({5: 0}, INVALID), ({5: (1 << 24) + 1}, INVALID), ({6: 48}, INVALID),
        ({6: 0}, INVALID), ({6: (1 << 17) + 32}, INVALID), ({8: 2}, INVALID), ({4: None}, INVALID),
        ({4: P + 2}, ALIGNMENT), ({0: None}, INVALID), ({2: P + 8}, ALIGNMENT), ({7: P + 2}, ALIGNMENT)])
    # x per_pair ids tokens topk E wq ws wg n k y dtype stream
    good = [P, 0, P, 4, 8, 64, P, P, P, 64, 256, P, 0, None]
    _refused(lib.fpq_moe_gemv_nvfp4, good, [
        ({1: 2}, INVALID), ({3: -1}, INVALID), ({3: 129}, INVALID), ({3: 1 << 40}, INVALID), ({4: 0}, INVALID),
        ({4: 33}, INVALID), ({5: 0}, INVALID), ({5: 1025}, INVALID), ({10: 16}, INVALID), ({8: None}, INVALID),
        ({2: None}, INVALID), ({6: P + 1}, ALIGNMENT)])


def test_no_device_is_unsupported(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; this checks the no-device path")
    assert lib.fpq_rmsnorm_quantize(0, P, 256, P, P, 4, 256, 1e-6, P, P, P, P, P, None) == UNSUPPORTED
    assert lib.fpq_rmsnorm_backward(P, P, 256, P, P, P, 4, 256, P, P, P, 1 << 30, None) == UNSUPPORTED
    assert lib.fpq_moe_gate(P, 1, P, 16, 64, 1, 8, 4, 2, 8, 1, 1.0, P, P, None) == UNSUPPORTED
    assert lib.fpq_moe_combine(P, 0, 128, P, P, 16, 8, 64, P, P, 0, None) == UNSUPPORTED
    assert lib.fpq_gemv_nvfp4(P, 4, P, P, P, 64, 256, P, 0, None) == UNSUPPORTED
    assert isinstance(lib.fpq_last_error_detail(), bytes) and ctypes.c_char_p


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_python_entry_points():
    """Wrong types and shapes, and tensors that are not on a GPU."""
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    x, w = _t(4, 256), _t(256)
    bad = [
        lambda: f.rmsnorm_quantize(_t(4, 256, dtype=f32), w),
        lambda: f.rmsnorm_quantize(_t(256), w),
        lambda: f.rmsnorm_quantize(_t(256, 4).T, w),
        lambda: f.rmsnorm_quantize(x, _t(128)),
        lambda: f.rmsnorm_quantize(x, _t(256, dtype=f32)),
        lambda: f.rmsnorm_quantize(x, w, residual=_t(4, 128)),
        lambda: f.rmsnorm_quantize(x, w, f.NVFP4),
        lambda: f.rmsnorm_quantize(_t(4, 40), _t(40), f.MXFP8),
        lambda: f.rmsnorm_quantize(x, w),                                            # not on a GPU
        lambda: f.rmsnorm_backward(_t(4, 128), x, w, _t(4, dtype=f32)),
        lambda: f.rmsnorm_backward(x, x, w, _t(4)),
        lambda: f.rmsnorm_backward(x, x, w, _t(5, dtype=f32)),
        lambda: f.rmsnorm_backward(x, x, w, _t(4, dtype=f32), dres=_t(4, 256, dtype=f32)),
        lambda: f.rmsnorm_backward(x, x, w, _t(4, dtype=f32)),
        lambda: moe.gate(_t(4, 8, dtype=torch.float16), 2),
        lambda: moe.gate(_t(8), 2),
        lambda: moe.gate(_t(4, 8), 2, bias=_t(8)),
        lambda: moe.gate(_t(4, 8), 2, bias=_t(4, dtype=f32)),
        lambda: moe.gate(_t(4, 8), 2),
        lambda: moe.gate_backward(_t(4, 2, dtype=f32), _t(4, 8), _t(4, 2, dtype=torch.int64)),
        lambda: moe.gate_backward(_t(4, 3, dtype=f32), _t(4, 8), _t(4, 2, dtype=i32)),
        lambda: moe.gate_backward(_t(4, 2, dtype=f32), _t(4, 8), _t(4, 2, dtype=i32)),
        lambda: moe.combine(_t(8, 64), _t(4, 2)),
        lambda: moe.combine(_t(8, 64), _t(4, 2, dtype=f32), rows=_t(4, 3, dtype=i32)),
        lambda: moe.combine(_t(2, 4, 64), _t(4, 2, dtype=f32)),
        lambda: moe.combine(_t(8, 64), _t(4, 2, dtype=f32), add=_t(4, 32)),
        lambda: moe.combine(_t(8, 64), _t(4, 2, dtype=f32), out_dtype=torch.float16),
        lambda: moe.combine(_t(8, 64), _t(4, 2, dtype=f32)),
        lambda: moe.combine_backward(_t(3, 64), _t(8, 64), _t(4, 2, dtype=f32)),
        lambda: moe.combine_backward(_t(4, 64), _t(8, 64), _t(4, 2, dtype=f32), dy=_t(8, 64, dtype=f32)),
        lambda: moe.combine_backward(_t(4, 64), _t(8, 64), _t(4, 2, dtype=f32)),
        lambda: moe.dispatch(_t(4, 64), _t(4, 2, dtype=i32), 8, rows=_t(4, 2, dtype=torch.int64)),
        lambda: f.gemv_nvfp4(_t(2, 64, dtype=f32), _t(8, 32, dtype=u8), _t(8, 4, dtype=u8), _t(1, dtype=f32)),
        lambda: f.gemv_nvfp4(_t(2, 64), _t(8, 16, dtype=u8), _t(8, 4, dtype=u8), _t(1, dtype=f32)),
        lambda: f.gemv_nvfp4(_t(2, 64), _t(8, 32, dtype=u8), _t(8, 2, dtype=u8), _t(1, dtype=f32)),
        lambda: f.gemv_nvfp4(_t(2, 64), _t(8, 32, dtype=u8), _t(8, 4, dtype=u8), _t(1, dtype=f32),
                             ids=_t(2, 2, dtype=i32)),
        lambda: f.gemv_nvfp4(_t(2, 64), _t(8, 32, dtype=u8), _t(8, 4, dtype=u8), _t(1, dtype=f32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")


def test_counts_whose_product_passes_64_bits(lib):
    far = 1 << 62
    assert lib.fpq_moe_gate(P, 1, P, far, 64, 1, 8, 4, 2, 8, 1, 1.0, P, P, None) == INVALID
    assert lib.fpq_moe_gate_backward(P, 0, P, P, far, 64, 0, 8, 1, 1.0, P, None) == INVALID
    assert lib.fpq_moe_combine(P, 0, 128, P, P, far, 8, 64, P, P, 0, None) == INVALID
    assert lib.fpq_moe_combine_backward(P, 1, P, 0, 128, P, P, far, 8, 64, P, P, None) == INVALID
    assert lib.fpq_moe_pair_rows(P, far, 8, 64, P, 1 << 30, P, P, None) == INVALID


def test_gate_backward_refuses_a_gradient_over_its_logits(lib):
    def call(logits, dlogits, dtype=0):
        return lib.fpq_moe_gate_backward(logits, dtype, P, P, 16, 64, 0, 8, 1, 1.0, dlogits, None)

    size = 16 * 64 * 2
    for dtype, n in ((0, size), (1, 2 * size)):
        for shift in (0, 16, n - 16):
            assert call(P, P + shift, dtype) == INVALID and b"overlap" in lib.fpq_last_error_detail()
            assert call(P + shift, P, dtype) == INVALID and b"overlap" in lib.fpq_last_error_detail()
    if not torch.cuda.is_available():                        # beside each other: as far as the device
        assert call(P, P + size) == UNSUPPORTED and call(P + size, P) == UNSUPPORTED


def test_combine_backward_of_every_row(lib):
    # dout dtype y dtype y_rows rows weights tokens topk hidden dy dweights ws wsb stream
    good = [P, 1, P, 0, 128, P, P, 16, 8, 64, P, P, P, 512, None]
    _refused(lib.fpq_moe_combine_backward_full, good, [
        ({1: 5}, INVALID), ({9: 4}, INVALID), ({5: None, 4: 100}, INVALID), ({0: None}, INVALID), ({10: None}, INVALID),
        ({11: None}, INVALID), ({5: P + 4}, ALIGNMENT), ({10: P + 8}, ALIGNMENT), ({12: None}, WORKSPACE),
        ({12: P + 4}, WORKSPACE), ({13: 511}, WORKSPACE), ({7: 0, 10: None}, INVALID)])
    assert lib.fpq_moe_combine_backward_full(*(good[:4] + [0] + good[5:7] + [0] + good[8:])) == 0     # nothing to write
