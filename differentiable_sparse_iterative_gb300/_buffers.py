"""Scratch buffers of the calls."""
from __future__ import annotations

from typing import Optional

import torch


def usable(ws: Optional[torch.Tensor], need: int, device) -> bool:
    """Whether the caller's workspace is there and holds `need` bytes.  Its address and size go to the kernels as
    they are, so one that is not dense memory of that device (a CPU tensor, a strided or an expanded view) raises."""
    if ws is None:
        return False
    if not ws.is_cuda or ws.get_device() != torch.device(device).index:
        raise ValueError(f"workspace must be a CUDA tensor on {device}, got {ws.device}")
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ws.numel() * ws.element_size() >= need
