"""Device buffers for one routed-expert MoE layer and the five-call chain.

PyTorch supplies device memory (torch.empty) and the stream; every step runs
in the HIP library through ``binding``.
"""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

from . import binding


@dataclasses.dataclass
class LayerBuffers:
    T: int
    E: int
    k: int
    H: int
    I: int
    topk_ids: torch.Tensor
    topk_weights: torch.Tensor
    bitmatrix: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    gather: torch.Tensor
    scatter: torch.Tensor
    y_sorted: torch.Tensor
    y: torch.Tensor
    ws: torch.Tensor

    @classmethod
    def allocate(cls, T, E, k, H, I, device="cuda"):
        return cls._allocate(T, E, k, H, I, device, binding.moe_workspace_bytes(T, E, k, H, I))

    @classmethod
    def allocate_fp8(cls, T, E, k, H, I, device="cuda"):
        """Buffers of a layer over block-scaled FP8 weights (run_layer_fp8)."""
        return cls._allocate(T, E, k, H, I, device, binding.moe_fp8_workspace_bytes(T, E, k, H, I))

    @classmethod
    def _allocate(cls, T, E, k, H, I, device, ws_bytes):
        dev = torch.device(device)
        if ws_bytes == 0:
            raise ValueError("invalid layer sizes")
        i32 = dict(dtype=torch.int32, device=dev)
        return cls(
            T, E, k, H, I,
            topk_ids=torch.empty((T, k), **i32),
            topk_weights=torch.empty((T, k), dtype=torch.float32, device=dev),
            bitmatrix=torch.empty((T, (E + 31) // 32), **i32),
            counts=torch.empty(E, **i32),
            offsets=torch.empty(E + 1, **i32),
            gather=torch.empty(T * k, **i32),
            scatter=torch.empty(T * k, **i32),
            y_sorted=torch.empty((T * k, H), dtype=torch.bfloat16, device=dev),
            y=torch.empty((T, H), dtype=torch.bfloat16, device=dev),
            ws=torch.empty(ws_bytes, dtype=torch.uint8, device=dev),
        )


def to_device(inp: dict, device="cuda") -> dict:
    """Copy one input dict (see inputs.make_inputs) to the GPU."""
    dev = torch.device(device)
    out = {}
    for key in ("logits", "x", "w1", "w1_s", "w2", "w2_s"):
        if key not in inp:
            continue
        a = np.ascontiguousarray(inp[key])
        if not a.flags.writeable:
            a = a.copy()
        if key == "x":
            a = a.view(np.int16)
        out[key] = torch.from_numpy(a).to(dev)
    if "x" in out:
        out["x"] = out["x"].view(torch.bfloat16)
    return out


def run_routing(dev: dict, b: LayerBuffers, stream=None, fused: bool = False):
    """A1-A3: three calls, or the fused front-end entry point (same outputs)."""
    if fused:
        binding.moe_route_and_group(dev["logits"], b.k, b.topk_ids, b.topk_weights, b.bitmatrix,
                                    b.counts, b.offsets, b.gather, b.scatter, b.ws, stream)
        return
    binding.moe_route(dev["logits"], b.k, b.topk_ids, b.topk_weights, stream)
    binding.moe_build_bitmatrix(b.topk_ids, b.E, b.bitmatrix, stream)
    binding.moe_expert_offsets(b.bitmatrix, b.topk_ids, b.E, b.counts, b.offsets, b.gather,
                               b.scatter, b.ws, stream)


def run_ffn(dev: dict, b: LayerBuffers, limit: float, stream=None):
    binding.moe_grouped_ffn_mxfp4(dev["x"], b.k, dev["w1"], dev["w1_s"], dev["w2"], dev["w2_s"],
                                  b.counts, b.offsets, b.gather, limit, b.y_sorted, b.ws, stream)
    binding.moe_combine(b.y_sorted, b.topk_weights, b.scatter, b.y, stream)


def run_layer(dev: dict, b: LayerBuffers, limit: float, stream=None, fused: bool = False):
    run_routing(dev, b, stream, fused)
    run_ffn(dev, b, limit, stream)


def run_forward(dev: dict, b: LayerBuffers, limit: float, stream=None):
    """The whole layer through the one-call entry point (same outputs as run_layer)."""
    binding.moe_forward_mxfp4(dev["logits"], dev["x"], b.k, dev["w1"], dev["w1_s"], dev["w2"],
                              dev["w2_s"], limit, b.topk_ids, b.topk_weights, b.bitmatrix,
                              b.counts, b.offsets, b.gather, b.scatter, b.y_sorted, b.y, b.ws,
                              stream)


def run_layer_fp8(dev: dict, b: LayerBuffers, limit: float, stream=None, **scoring):
    """The layer over block-scaled FP8 expert weights with scored routing (`scoring`: the
    keyword arguments of binding.moe_route_scored): route and group, grouped FFN, combine."""
    binding.moe_route_scored_and_group(dev["logits"], b.k, b.topk_ids, b.topk_weights, b.bitmatrix,
                                       b.counts, b.offsets, b.gather, b.scatter, b.ws,
                                       stream=stream, **scoring)
    binding.moe_grouped_ffn_fp8(dev["x"], b.k, dev["w1"], dev["w1_s"], dev["w2"], dev["w2_s"],
                                b.counts, b.offsets, b.gather, limit, b.y_sorted, b.ws, stream)
    binding.moe_combine(b.y_sorted, b.topk_weights, b.scatter, b.y, stream)


@dataclasses.dataclass
class BlockBuffers:
    """Buffers of run_block_fp8: the layer's, the norm's outputs, the router's logits, the shared
    projection's result, and the batch's rows by adapter (L = 0: no adapters)."""
    layer: LayerBuffers
    sum: torch.Tensor
    h: torch.Tensor
    hq: torch.Tensor
    hs: torch.Tensor
    logits: torch.Tensor
    shared: torch.Tensor
    adapter_offsets: torch.Tensor
    adapter_rows: torch.Tensor
    lora_ws: torch.Tensor

    @classmethod
    def allocate_fp8(cls, T, E, k, H, I, N, L=0, R=8, device="cuda"):
        dev = torch.device(device)

        def new(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device=dev)

        ws = max(binding.moe_lora_add_workspace_bytes(T, n, H, R, L) for n in (E, N)) if L else 0
        return cls(LayerBuffers.allocate_fp8(T, E, k, H, I, device), sum=new(T, H), h=new(T, H),
                   hq=new(T, H, dtype=torch.float8_e4m3fn), hs=new(T, (H + 127) // 128, dtype=torch.float32),
                   logits=new(T, E, dtype=torch.float32), shared=new(T, N),
                   adapter_offsets=new(L + 1, dtype=torch.int32), adapter_rows=new(T, dtype=torch.int32),
                   lora_ws=new(ws, dtype=torch.uint8))


def run_block_fp8(dev: dict, b: BlockBuffers, limit: float, eps: float = 1e-6, stream=None, **scoring):
    """The layer with what stands around it: residual addition and norm (bf16 for the experts, FP8 for
    the dense products), the router's product and a shared projection beside the experts, each with
    the requests' adapters if dev["adapter"] is given, then run_layer_fp8 on the routed rows.

    dev: x, residual [T, H], norm [H], router [E, H] and shared [N, H] in block-scaled FP8 with
    router_s and shared_s, w1, w1_s, w2, w2_s; with adapters adapter [T], scaling [L] or None, and
    router_a, router_b, shared_a, shared_b.  Leaves the stream in b.sum, the experts' sum in
    b.layer.y and the projection in b.shared."""
    binding.moe_rms_norm(dev["x"], dev["norm"], eps, residual=dev["residual"], sum=b.sum, y=b.h, q=b.hq,
                         scale=b.hs, stream=stream)
    binding.moe_gemm_fp8(b.hq, b.hs, dev["router"], dev["router_s"], b.logits, stream=stream)
    binding.moe_gemm_fp8(b.hq, b.hs, dev["shared"], dev["shared_s"], b.shared, stream=stream)
    if dev.get("adapter") is not None:
        binding.moe_lora_group(dev["adapter"], dev["router_a"].shape[0], b.adapter_offsets, b.adapter_rows, stream)
        for name, y in (("router", b.logits), ("shared", b.shared)):
            binding.moe_lora_add(b.h, dev[name + "_a"], dev[name + "_b"], dev.get("scaling"), b.adapter_offsets,
                                 b.adapter_rows, y, y, b.lora_ws, stream)
    run_layer_fp8(dict(dev, x=b.h, logits=b.logits), b.layer, limit, stream, **scoring)


def bf16_tensor_to_f32(t: torch.Tensor) -> np.ndarray:
    """Exact bf16 -> fp32 on the host (for comparisons)."""
    return t.float().cpu().numpy()
