"""The Python binding of scored routing and the FP8 operators (CPU: no call reaches the library)."""
from __future__ import annotations

import pytest
import torch

from mxfp4_routed_expert_route_amd import binding


def _calls():
    """One call of each entry point, on CPU tensors of the right types and shapes."""
    T, E, k, H, I = 4, 8, 2, 128, 128
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    f32, bf16 = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    logits = (f32(T, E), bf16(T, E))
    for l in logits:
        yield lambda l=l: binding.moe_route_scored(l, k, i32(T, k), f32(T, k), bias=f32(E))
        yield lambda l=l: binding.moe_route_scored_and_group(l, k, i32(T, k), f32(T, k), i32(T, 1), i32(E), i32(E + 1),
                                                             i32(T * k), i32(T * k), u8(64))
    yield lambda: binding.moe_quantize_fp8(bf16(T, H), u8(T, H), f32(T, 1))
    yield lambda: binding.moe_gemm_fp8(u8(T, H), f32(T, 1), u8(I, H), f32(1, 1), bf16(T, I), u8(16))
    yield lambda: binding.moe_gemm_fp8(u8(T, H), f32(T, 1), u8(I, H), f32(1, 1), f32(T, I))
    yield lambda: binding.moe_grouped_ffn_fp8(bf16(T, H), k, u8(E, 2 * I, H), f32(E, 2, 1), u8(E, H, I), f32(E, 1, 1),
                                              i32(E), i32(E + 1), i32(T * k), 10.0, bf16(T * k, H), u8(64))


def test_every_argument_is_given_to_the_native_checks_as_they_take_it(monkeypatch):
    # the native check takes a tuple of types and a tuple shape; anything else goes the slow way
    seen = []

    def arg(t, dtypes, shape, dev, name):
        assert isinstance(dtypes, tuple) and isinstance(shape, tuple), name
        assert t.dtype in dtypes and tuple(t.shape) == shape, name
        seen.append(name)
        return 0

    monkeypatch.setattr(binding, "_arg", arg)
    monkeypatch.setattr(binding, "_run", lambda *a: None)
    for call in _calls():
        call()
    assert seen.count("logits") == 4 and len(seen) == 2 * 4 + 2 * 9 + 3 + 6 + 5 + 10


@pytest.mark.parametrize("name", ["groups", "topk_groups", "group_top"])
@pytest.mark.parametrize("value", [2 ** 32 + 1, -2 ** 32 + 1, 2 ** 31, -2 ** 31 - 1])
def test_numbers_past_32_bits_are_refused(name, value):
    # the C interface takes 32-bit sizes, and ctypes cuts a larger one down without a word
    logits = torch.zeros(2, 8)
    out = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    with pytest.raises(ValueError, match=name):
        binding.moe_route_scored(logits, 2, *out, **{name: value})


def test_shapes_past_32_bits_are_refused():
    # shapes alone (no memory); 2^32 + 128 would arrive as 128
    big = 2 ** 32 + 128
    meta = lambda *s, dtype=torch.uint8: torch.empty(s, dtype=dtype, device="meta")
    f32 = lambda *s: meta(*s, dtype=torch.float32)
    i32 = lambda *s: meta(*s, dtype=torch.int32)
    bf16 = lambda *s: meta(*s, dtype=torch.bfloat16)
    for call, match in (
            (lambda: binding.moe_route_scored(f32(1, big), 2, i32(1, 2), f32(1, 2)), "E = "),
            (lambda: binding.moe_route_scored(f32(1, 8), big, i32(1, big), f32(1, big)), "k = "),
            (lambda: binding.moe_route_scored_and_group(f32(1, big), 2, i32(1, 2), f32(1, 2), i32(1, big // 32), i32(big),
                                                        i32(big + 1), i32(2), i32(2), meta(64)), "E = "),
            (lambda: binding.moe_quantize_fp8(bf16(1, big), meta(1, big), f32(1, big // 128)), "K = "),
            (lambda: binding.moe_gemm_fp8(meta(1, big), f32(1, big // 128), meta(1, big), f32(1, big // 128), f32(1, 1)), "K = "),
            (lambda: binding.moe_gemm_fp8(meta(1, 128), f32(1, 1), meta(big, 128), f32(big // 128, 1), f32(1, big)), "N = "),
            (lambda: binding.moe_grouped_ffn_fp8(bf16(1, big), 1, meta(1, 256, big), f32(1, 2, big // 128), meta(1, big, 128),
                                                 f32(1, big // 128, 1), i32(1), i32(2), i32(1), 0.0, bf16(1, big), meta(64)), "H = "),
            (lambda: binding.moe_grouped_ffn_fp8(bf16(1, 128), 1, meta(1, 2 * big, 128), f32(1, big // 64, 1), meta(1, 128, big),
                                                 f32(1, 1, big // 128), i32(1), i32(2), i32(1), 0.0, bf16(1, 128), meta(64)), "I = "),
            (lambda: binding.moe_grouped_ffn_fp8(bf16(1, 128), 1, meta(big, 256, 128), f32(big, 2, 1), meta(big, 128, 128),
                                                 f32(big, 1, 1), i32(big), i32(big + 1), i32(1), 0.0, bf16(1, 128), meta(64)), "E = "),
            (lambda: binding.moe_grouped_ffn_fp8(bf16(1, 128), big, meta(4, 256, 128), f32(4, 2, 1), meta(4, 128, 128),
                                                 f32(4, 1, 1), i32(4), i32(5), i32(big), 0.0, bf16(big, 128), meta(64)), "k = ")):
        with pytest.raises(ValueError, match=match):
            call()
    # sizes are checked by the calls that ask for a workspace too: none for what no call takes
    assert binding.moe_fp8_workspace_bytes(16, big, 6, 4096, 2048) == 0
    assert binding.moe_fp8_workspace_bytes(16, 256, 6, big, 2048) == 0
    assert binding.moe_fp8_workspace_bytes(2 ** 64 + 16, 256, 6, 4096, 2048) == 0
    assert binding.moe_gemm_fp8_workspace_bytes(4, big, 128) == 0


def test_the_fp8_layer_runs_on_its_tensors_gpu(monkeypatch):
    # tensors on GPU 1 while GPU 0 is current: every call of the layer goes to GPU 1's stream
    import contextlib
    import dataclasses

    from mxfp4_routed_expert_route_amd import layer

    T, E, k, H, I = 4, 8, 2, 128, 128

    class OnGpu1:
        """A tensor's face, as the binding looks at it."""
        is_cuda = True

        def __init__(self, dtype, *shape):
            self.dtype, self.shape = dtype, torch.Size(shape)

        def dim(self):
            return len(self.shape)

        def numel(self):
            return self.shape.numel()

        def get_device(self):
            return 1

        device = property(lambda self: torch.device("cuda", 1))

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 4096

    i32, f32, bf16, u8 = (lambda *s, d=d: OnGpu1(d, *s) for d in (torch.int32, torch.float32, torch.bfloat16, torch.uint8))
    b = layer.LayerBuffers(T, E, k, H, I, i32(T, k), f32(T, k), i32(T, 1), i32(E), i32(E + 1), i32(T * k), i32(T * k),
                           bf16(T * k, H), bf16(T, H), u8(1 << 16))
    assert len(dataclasses.fields(b)) == 15
    dev = dict(logits=f32(T, E), x=bf16(T, H), w1=u8(E, 2 * I, H), w1_s=f32(E, 2, 1), w2=u8(E, H, I), w2_s=f32(E, 1, 1))
    current, calls = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d
        yield
        current[0] = before

    class Stream:
        def __init__(self, dev):
            self.cuda_stream = 1000 + dev

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, current[0], a[-1])) or 0

    monkeypatch.setattr(binding, "_arg", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(binding, "load", Lib)
    monkeypatch.setattr(binding, "_fns", {})
    monkeypatch.setattr(binding, "_several", None)
    monkeypatch.setattr(binding, "_raw_stream", lambda dev: 1000 + dev)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: Stream(current[0] if dev is None else dev))
    monkeypatch.setattr(torch.cuda, "device", device)
    layer.run_layer_fp8(dev, b, 10.0)
    assert calls == [(n, 1, 1001) for n in ("moe_route_scored_and_group", "moe_grouped_ffn_fp8", "moe_combine")]
    calls.clear()
    layer.run_layer_fp8(dev, b, 10.0, stream=77)
    assert calls == [(n, 1, 77) for n in ("moe_route_scored_and_group", "moe_grouped_ffn_fp8", "moe_combine")]
    assert current == [0]
