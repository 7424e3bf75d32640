"""CPU checks of the host side of the norm, the few-token expert layer and NVFP4
storage and products: every refusal comes back as a status (or a Python
exception) before anything is enqueued."""
import pytest
import torch

from ffn_gated_activation_b200 import abi, block

OK, INVALID, UNSUP, MISAL = abi.SITU_OK, abi.SITU_ERR_INVALID_ARG, abi.SITU_ERR_UNSUPPORTED, abi.SITU_ERR_MISALIGNED
# Fake, well-separated, 256-byte-aligned device addresses: validation never dereferences them.
P = [0x1000_0000 * k for k in range(0, 14)]

BASE = {
    "norm": (abi.situ_glu_rms_norm_fwd, dict(
        x=P[1], dtype=0, tokens=8, hidden=256, x_row_stride=256, residual=P[2], residual_row_stride=256, weight=P[3],
        weight_dtype=1, epsilon=1e-6, h=P[4], h_row_stride=256, y=P[5], y_row_stride=256, stream=None)),
    "norm_mx": (abi.situ_glu_rms_norm_fwd_mxfp8, dict(
        x=P[1], dtype=0, tokens=8, hidden=256, x_row_stride=256, residual=None, residual_row_stride=0, weight=P[3],
        weight_dtype=0, epsilon=1e-6, h=None, h_row_stride=0, y_data=P[5], y_data_row_stride=256, y_scale=P[6],
        y_scale_row_stride=8, rule=0, stream=None)),
    "norm_bwd": (abi.situ_glu_rms_norm_bwd, dict(
        grad_y=P[1], grad_y_row_stride=256, grad_h=P[2], grad_h_row_stride=256, h=P[3], dtype=0, tokens=8, hidden=256,
        h_row_stride=256, weight=P[4], weight_dtype=0, epsilon=1e-6, d_x=P[5], d_x_row_stride=256, d_weight=P[6],
        workspace=P[7], workspace_bytes=8 * 256 * 4, stream=None)),
    "moe": (abi.situ_glu_moe_fwd, dict(
        x=P[1], tokens=4, hidden=256, x_row_stride=256, topk_ids=P[2], topk=2, topk_ids_row_stride=2, topk_weights=P[3],
        weights_dtype=1, topk_weights_row_stride=2, w1=P[4], experts=4, inter=128, w1_row_stride=256, w2=P[5],
        w2_row_stride=128, beta=4.0, has_linear_beta=1, linear_beta=25.0, y=P[6], y_row_stride=256, workspace=P[7],
        workspace_bytes=1 << 20, stream=None)),
    "quantize": (abi.situ_glu_nvfp4_quantize, dict(
        x=P[1], dtype=0, rows=8, cols=64, x_row_stride=64, data=P[2], data_row_stride=32, scale=P[3], scale_row_stride=4,
        amax=P[4], amax_given=1, stream=None)),
    "dequantize": (abi.situ_glu_nvfp4_dequantize, dict(
        data=P[1], data_row_stride=32, scale=P[2], scale_row_stride=4, amax=P[3], rows=8, cols=64, out=P[4], dtype=0,
        out_row_stride=64, stream=None)),
    "gemm": (abi.situ_glu_nvfp4_gemm, dict(
        a_data=P[1], a_data_row_stride=64, a_scale=P[2], a_scale_row_stride=8, a_amax=P[3], tokens=8, k=128, w_data=P[4],
        w_data_row_stride=64, w_scale=P[5], w_scale_row_stride=8, w_amax=P[6], w_amax_stride=1, experts=3, n=64,
        offsets=P[7], out=P[8], out_dtype=0, out_row_stride=64, stream=None)),
}

CASES = [
    ("norm", dict(dtype=5), INVALID), ("norm", dict(weight_dtype=2), INVALID), ("norm", dict(tokens=-1), INVALID),
    ("norm", dict(hidden=0), INVALID), ("norm", dict(hidden=252), MISAL), ("norm", dict(hidden=32776), UNSUP),
    ("norm", dict(dtype=1, hidden=16388), UNSUP), ("norm", dict(epsilon=-1.0), INVALID),
    ("norm", dict(epsilon=float("nan")), INVALID), ("norm", dict(x_row_stride=248), INVALID),
    ("norm", dict(residual_row_stride=255), INVALID), ("norm", dict(h=None), INVALID),
    ("norm", dict(residual=None), INVALID), ("norm", dict(x=None), INVALID), ("norm", dict(y=None), INVALID),
    ("norm", dict(weight=None), INVALID), ("norm", dict(weight=P[3] + 8), MISAL), ("norm", dict(x=P[1] + 8), MISAL),
    ("norm", dict(y_row_stride=260), MISAL), ("norm", dict(h=P[1]), INVALID), ("norm", dict(y=P[4] + 16), INVALID),
    ("norm", dict(y=P[3]), INVALID), ("norm", dict(tokens=1 << 62), INVALID), ("norm", dict(h_row_stride=200), INVALID),
    ("norm", dict(tokens=0, x=None, y=None, h=P[4]), OK),
    ("norm_mx", dict(hidden=48, x_row_stride=48, y_data_row_stride=48), INVALID), ("norm_mx", dict(rule=2), INVALID),
    ("norm_mx", dict(y_scale_row_stride=7), INVALID), ("norm_mx", dict(y_data_row_stride=255), INVALID),
    ("norm_mx", dict(y_scale=None), INVALID), ("norm_mx", dict(y_data=P[5] + 4), MISAL),
    ("norm_mx", dict(y_scale=P[5] + 100), INVALID), ("norm_mx", dict(tokens=0), OK),
    ("norm_bwd", dict(workspace=None), INVALID), ("norm_bwd", dict(workspace_bytes=8191), INVALID),
    ("norm_bwd", dict(workspace=P[7] + 8), MISAL), ("norm_bwd", dict(d_x=P[1]), INVALID),
    ("norm_bwd", dict(d_weight=P[6] + 1), MISAL), ("norm_bwd", dict(h=None), INVALID),
    ("norm_bwd", dict(grad_y=None), INVALID), ("norm_bwd", dict(grad_h_row_stride=100), INVALID),
    ("norm_bwd", dict(d_weight=P[7]), INVALID), ("norm_bwd", dict(tokens=0, d_weight=None), OK),
    ("moe", dict(tokens=65), UNSUP), ("moe", dict(tokens=-1), INVALID), ("moe", dict(topk=0), UNSUP),
    ("moe", dict(topk=17, topk_ids_row_stride=17, topk_weights_row_stride=17), UNSUP), ("moe", dict(experts=0), UNSUP),
    ("moe", dict(experts=1025), UNSUP), ("moe", dict(hidden=224, x_row_stride=224), UNSUP),
    ("moe", dict(inter=96, w2_row_stride=96), UNSUP), ("moe", dict(inter=0), UNSUP), ("moe", dict(beta=0.0), INVALID),
    ("moe", dict(has_linear_beta=2), INVALID), ("moe", dict(linear_beta=float("inf")), INVALID),
    ("moe", dict(weights_dtype=4), INVALID), ("moe", dict(topk_ids_row_stride=1), INVALID),
    ("moe", dict(topk_weights_row_stride=1), INVALID), ("moe", dict(w1_row_stride=128), INVALID),
    ("moe", dict(w2_row_stride=64), INVALID), ("moe", dict(x=None), INVALID), ("moe", dict(topk_ids=None), INVALID),
    ("moe", dict(workspace=None), INVALID), ("moe", dict(workspace_bytes=100), INVALID),
    ("moe", dict(workspace=P[7] + 8), MISAL), ("moe", dict(x=P[1] + 2), MISAL), ("moe", dict(topk_ids=P[2] + 4), MISAL),
    ("moe", dict(topk_weights=P[3] + 2), MISAL), ("moe", dict(y=P[1]), INVALID), ("moe", dict(workspace=P[4]), INVALID),
    ("moe", dict(y=P[7]), INVALID), ("moe", dict(w1_row_stride=1 << 62), INVALID), ("moe", dict(tokens=0), OK),
    ("quantize", dict(cols=40), INVALID), ("quantize", dict(cols=0), INVALID), ("quantize", dict(rows=-1), INVALID),
    ("quantize", dict(amax_given=3), INVALID), ("quantize", dict(amax=None), INVALID),
    ("quantize", dict(amax=P[4] + 2), MISAL), ("quantize", dict(data=None), INVALID), ("quantize", dict(x=None), INVALID),
    ("quantize", dict(data=P[2] + 4), MISAL), ("quantize", dict(data_row_stride=36), MISAL),
    ("quantize", dict(data_row_stride=24), INVALID), ("quantize", dict(scale_row_stride=3), INVALID),
    ("quantize", dict(x_row_stride=68), MISAL), ("quantize", dict(scale=P[2] + 8), INVALID),
    ("quantize", dict(data=P[1]), INVALID), ("quantize", dict(amax=P[1]), INVALID), ("quantize", dict(dtype=9), INVALID),
    ("quantize", dict(rows=1 << 62), INVALID), ("quantize", dict(rows=0), OK),
    ("dequantize", dict(out=P[4] + 8), MISAL), ("dequantize", dict(out=None), INVALID),
    ("dequantize", dict(amax=None), INVALID), ("dequantize", dict(out=P[1]), INVALID),
    ("dequantize", dict(data=P[1] + 4), MISAL), ("dequantize", dict(cols=8), INVALID), ("dequantize", dict(rows=0), OK),
    ("gemm", dict(k=96), UNSUP), ("gemm", dict(k=0), UNSUP), ("gemm", dict(n=60), UNSUP), ("gemm", dict(n=0), UNSUP),
    ("gemm", dict(experts=0), UNSUP), ("gemm", dict(experts=1025), UNSUP), ("gemm", dict(tokens=-1), INVALID),
    ("gemm", dict(tokens=1 << 31), UNSUP), ("gemm", dict(offsets=None), INVALID), ("gemm", dict(out_dtype=3), INVALID),
    ("gemm", dict(a_data_row_stride=48), INVALID), ("gemm", dict(a_scale_row_stride=4), INVALID),
    ("gemm", dict(w_scale_row_stride=10), MISAL), ("gemm", dict(w_data_row_stride=72), MISAL),
    ("gemm", dict(a_data=P[1] + 8), MISAL), ("gemm", dict(a_scale=P[2] + 2), MISAL), ("gemm", dict(out=P[8] + 4), MISAL),
    ("gemm", dict(out_row_stride=68), MISAL), ("gemm", dict(out_row_stride=56), INVALID),
    ("gemm", dict(a_amax=None), INVALID), ("gemm", dict(w_amax=None), INVALID), ("gemm", dict(w_amax_stride=-1), INVALID),
    ("gemm", dict(out=P[1]), INVALID), ("gemm", dict(out=P[7]), INVALID), ("gemm", dict(w_data=None), INVALID),
    ("gemm", dict(offsets=P[7] + 4), MISAL), ("gemm", dict(tokens=0), OK),
]


@pytest.mark.parametrize("entry,change,status", CASES, ids=[f"{e}-{'-'.join(c)}-{i}" for i, (e, c, _) in enumerate(CASES)])
def test_arguments_are_validated_on_the_host(entry, change, status, native_lib_path):
    call, args = BASE[entry]
    if entry == "quantize" and change == dict(rows=0):
        change = dict(rows=0, amax_given=1)  # a given maximum: nothing at all to enqueue
    assert call(**{**args, **change}) == status, abi.situ_glu_last_error()
    if status != OK:
        assert abi.situ_glu_last_error()


def test_workspace_queries(native_lib_path):
    q = abi.situ_glu_rms_norm_bwd_workspace_bytes
    assert q(8, 256, 1) == 8 * 256 * 4 and q(8, 256, 0) == 0 and q(0, 256, 1) == 0 and q(-3, 256, 1) == 0
    assert q(100_000, 7168, 1) == 148 * 7168 * 4  # one row of sums per chunk, at most 148 chunks
    assert q(8, 1 << 20, 1) == 0
    m = abi.situ_glu_moe_workspace_bytes
    assert m(1, 8, 7168, 2048) == 8 * 2048 * 4 + 8 * 7168 * 4 + 256
    assert m(65, 8, 7168, 2048) == 0 and m(0, 8, 64, 64) == 0 and m(1, 17, 64, 64) == 0


@pytest.mark.parametrize("call", [
    lambda t: block.situ_glu_rms_norm_fwd(t(4, 64), t(64)),
    lambda t: block.situ_glu_rms_norm_fwd_mxfp8(t(4, 64), t(64)),
    lambda t: block.situ_glu_rms_norm_bwd(t(4, 64), t(4, 64), t(64)),
    lambda t: block.add_rms_norm(t(4, 64), t(64)),
    lambda t: block.situ_glu_moe_fwd(t(2, 64), torch.zeros(2, 1, dtype=torch.int64), None, t(2, 128, 64), t(2, 64, 64)),
    lambda t: block.situ_glu_nvfp4_quantize(t(4, 64)),
], ids=["fwd", "fwd_mxfp8", "bwd", "autograd", "moe", "quantize"])
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(lambda *s: torch.zeros(*s, dtype=torch.bfloat16))


def test_matrix_views_are_copied_only_where_rows_are_not_runs():
    t = torch.arange(48.0).reshape(4, 12)
    m, pitch = block._matrix(t[:, 2:8], 6)
    assert m.data_ptr() == t[:, 2:8].data_ptr() and pitch == 12
    assert block._matrix(t.t(), 4)[0].is_contiguous()
    m, pitch = block._matrix(t[:1].expand(4, 12), 12)  # overlapping rows
    assert m.stride(0) == 12 and pitch == 12
    assert block._matrix(t[:0], 12)[0].shape == (0, 12)
    wide = torch.zeros(2, 3, 12)
    assert block._matrix(wide, 12) == (wide, 12) and block._rows(wide, 12) == 6  # contiguous: as it is
    assert block._matrix(wide[:, :, :8], 8)[0].shape == (6, 8) and block._rows(wide[:0], 12) == 0
    assert block._matrix(t[1:2, 3:9], 6)[1] == 6  # one row: its pitch is its width


def test_outputs_of_the_wrong_shape_are_refused():
    with pytest.raises(ValueError, match="shape"):
        block._out(torch.empty(3, 4), (3, 5), torch.float32, torch.device("cpu"), "out")
    with pytest.raises(TypeError, match="one-byte"):
        block._bytes(torch.empty(3, 4), (3, 4), torch.uint8, torch.device("cpu"), "codes")
    o, o2, pitch = block._out(torch.empty(3, 9)[:, :4], (3, 4), torch.float32, torch.device("cpu"), "out")
    assert o2.data_ptr() == o.data_ptr() and pitch == 9
