"""What the Python binding of the microscaled-format calls decides from its tensors alone (no GPU needed: host and meta
tensors are refused later than these are, by another message)."""

import pytest
import torch

import mixture_experts_ffn_infer_gb300 as mx


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_ffn_infer_gb300 import build
    build.build()


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


# ---------------------------------------------------------------- rows that share memory

@pytest.mark.parametrize("residual", [bf16(1, 64).expand(5, 64), bf16(5 * 32 + 32).as_strided((5, 64), (32, 1))])
@pytest.mark.parametrize("sum_out", [None, bf16(5, 64), bf16(1, 64).expand(5, 64)])
def test_a_residual_whose_rows_overlap_is_refused(residual, sum_out):
    with pytest.raises(ValueError, match="residual: .*rows of their own"):
        mx.mx_add_rmsnorm(bf16(5, 64), residual, bf16(64), 1e-6, 1, sum_out=sum_out)


def test_other_rows_that_overlap_are_refused():
    x, gain, shared = bf16(5, 64), bf16(64), bf16(1, 64).expand(5, 64)
    with pytest.raises(ValueError, match="x: .*rows of their own"):
        mx.mx_quantise(shared, 1)
    with pytest.raises(ValueError, match="x: .*rows of their own"):
        mx.mx_add_rmsnorm(shared, x, gain, 1e-6, 1)
    with pytest.raises(ValueError, match="sum_out: .*rows of their own"):
        mx.mx_add_rmsnorm(x, None, gain, 1e-6, 1, sum_out=shared)


def test_the_row_strides_of_residual_and_sum_have_to_agree():
    with pytest.raises(ValueError, match="row stride differs"):
        mx.mx_add_rmsnorm(bf16(5, 64), bf16(5, 128)[:, :64], bf16(64), 1e-6, 1, sum_out=bf16(5, 64))


# ---------------------------------------------------------------- where rows go

@pytest.mark.parametrize("fmt", range(4))
def test_fewer_rows_than_x_are_refused_without_positions(fmt):
    x, gain, few = bf16(5, 64), bf16(64), mx.mx_rows(fmt, 4, 64, "cpu")
    for call in (lambda: mx.mx_quantise(x, fmt, out=few), lambda: mx.mx_quantise(x, fmt, out_rows=4),
                 lambda: mx.mx_add_rmsnorm(x, x, gain, 1e-6, fmt, out=few),
                 lambda: mx.mx_add_rmsnorm(x, x, gain, 1e-6, fmt, out_rows=4)):
        with pytest.raises(ValueError, match="fewer rows than x, and no positions"):
            call()
    for call in (lambda: mx.mx_quantise(x, fmt, out=mx.mx_rows(fmt, 6, 64, "cpu")),          # more is room to spare
                 lambda: mx.mx_quantise(x, fmt, positions=torch.zeros(5, 1, dtype=torch.int32), out_rows=4)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_a_refused_call_leaves_the_factor_of_out():
    x, gain, old, new = bf16(5, 64), bf16(64), torch.ones(1), torch.full((1,), 2.0)
    out = mx.mx_rows(3, 5, 64, "cpu", global_scale=old)
    h = mx.mx_rows(3, 5, 64, "cpu", global_scale=old)
    w = mx.MxWeights(3, 1, 64, 64, torch.zeros(mx.moe_mx_packed_bytes(mx.moe_mx_weights(3, 1, 64, 64, 1, None, None, None)),
                                               dtype=torch.uint8), swiglu=True)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: mx.mx_quantise(x, 3, global_scale=new, out=out),
                 lambda: mx.mx_add_rmsnorm(x, x, gain, 1e-6, 3, global_scale=new, out=out),
                 lambda: mx.mx_add_rmsnorm(x, x, gain, 1e-6, 3, out=out),
                 lambda: mx.mx_grouped_swiglu(h, w, off, h_global=new, out=out)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
        assert out.global_scale is old


# ---------------------------------------------------------------- sizes past 32 bits

def test_sizes_past_32_bits_are_unsupported():
    wide = (1 << 32) + 64                    # cut to 32 bits: 64, which would be done without a word
    x = torch.empty(1, wide, dtype=torch.bfloat16, device="meta")
    gain = torch.empty(wide, dtype=torch.bfloat16, device="meta")
    rows = mx.MxRows(0, wide, torch.empty(1, 2 * wide, dtype=torch.uint8, device="meta"))
    ids = torch.empty(1, wide, dtype=torch.int32, device="meta")
    few = torch.empty(1, 64, dtype=torch.bfloat16, device="meta")
    for call in (lambda: mx.mx_quantise(x, 0), lambda: mx.mx_add_rmsnorm(x, None, gain, 1e-6, 0),
                 lambda: mx.mx_dequantise(rows), lambda: mx.mx_quantise(few, 0, positions=ids),
                 lambda: mx.mx_layer_forward(few, None, None, 0.0, ids, ids.float(), None, None)):
        with pytest.raises(mx.MoeError):
            call()
    w = mx.MxWeights(0, 1, 64, 64, torch.empty(32768, dtype=torch.uint8, device="meta"))
    r = mx.MxRows(0, 64, torch.empty(1, 128, dtype=torch.uint8, device="meta"))
    off = torch.empty(2, dtype=torch.int32, device="meta")
    with pytest.raises(mx.MoeError):
        mx.mx_grouped_product(r, w, off, out_type=1 << 32)


# ---------------------------------------------------------------- the stream argument

class Here:
    """A tensor's place, without the device."""

    def __init__(self, index):
        self.device = torch.device("cuda", index)


class Stream:
    cuda_stream = 77

    def __init__(self, index):
        self.device = torch.device("cuda", index)


@pytest.fixture
def made(monkeypatch):
    """Streams that _on makes and makes current, by fakes of torch's."""
    import contextlib
    log = []

    def external(handle, device=None):
        s = Stream(0 if device is None else device.index)       # torch's default is the current device, 0 here
        log.append(("external", handle, s.device.index))
        return s

    @contextlib.contextmanager
    def current(s):
        log.append(("current", s.device.index))
        yield

    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: log.append(("default", device.index)) or Stream(device.index))
    monkeypatch.setattr(torch.cuda, "stream", current)
    return log


def test_a_stream_handle_is_of_the_tensors_device(made):
    from mixture_experts_ffn_infer_gb300.mx import _on
    for first in (Here(1), mx.MxRows(1, 64, Here(1))):
        assert _on(4096, lambda *a: len(a), first, None) == 2
        assert made == [("external", 4096, 1), ("current", 1)]
        made.clear()


def test_stream_zero_is_the_default_stream(made):
    # (an ExternalStream of handle 0 would be a new stream of torch's pool)
    from mixture_experts_ffn_infer_gb300.mx import _on
    _on(0, lambda *a: None, Here(1))
    assert made == [("default", 1), ("current", 1)]


def test_a_stream_of_another_device_is_refused(made):
    from mixture_experts_ffn_infer_gb300.mx import _on
    with pytest.raises(ValueError, match="stream: of cuda:0, the tensors are on cuda:1"):
        _on(Stream(0), lambda *a: pytest.fail("called"), Here(1))
    assert _on(Stream(1), lambda *a: 5, Here(1)) == 5 and made == [("current", 1)]


def test_refusals_come_with_a_stream_too():
    with pytest.raises(ValueError, match="CUDA"):
        mx.mx_quantise(bf16(5, 64), 1, stream=0)
    with pytest.raises(ValueError, match="x: expected a tensor"):
        mx.mx_quantise(None, 1, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        mx.mx_pack(mx.mx_rows(1, 4, 64, "cpu"), 1, stream=4096)
