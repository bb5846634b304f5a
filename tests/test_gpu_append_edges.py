"""Scales whose quotients lie next to the border between two e4m3 values: the
codes are those of the division, bit for bit."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from test_gpu_paged import Case

pytestmark = pytest.mark.gpu


def _scales():
    """fp32 scales that take a power of two next to a border, within 4 steps, and those just below a power of two."""
    borders = [(1 + (2 * k + 1) / 16) * 2.0 ** e for k in range(8) for e in (-6, 0)] + [(2 * k + 1) * 2.0 ** -10 for k in range(8)]
    near = np.array([1.0 / b for b in borders], np.float32).view(np.int32)
    s = (near[:, None] + np.arange(-4, 5)[None]).astype(np.int32).view(np.float32).ravel()
    ones = np.array([(2 - 2.0 ** -23) * 2.0 ** e for e in (-59, -21, -3, 2, 9, 40)], np.float32)
    return np.concatenate([s, ones, s[:(-len(s) - len(ones)) % 8]])


def test_append_quotients_next_to_a_border():
    c = Case([(64, 64)], 8, 8, 128, 16, "fp8", poison=False)
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).to(DEV)
    # each bf16 pattern meets one scale of eight a turn: turn the patterns over the heads
    pages = torch.from_numpy(c.table[0, :4]).to(DEV)
    scales = torch.from_numpy(_scales()).to(DEV).view(-1, 8)
    for i, row in enumerate(scales):
        say(f"append borders {i}")
        for t in range(8):
            c.new_k = every.view(64, 8, 128).roll(t, dims=1).contiguous()
            c.new_v = c.new_k.flip(0).contiguous()
            c.k_scale, c.v_scale = row.contiguous(), row.flip(0).contiguous()
            c.append()
            torch.cuda.synchronize()
            k = c.k[pages].view(torch.uint8).permute(0, 2, 1, 3).reshape(64, 8, 128)
            v = c.v[pages].view(torch.uint8).permute(0, 3, 1, 2).reshape(64, 8, 128)
            for got, x, scale in ((k, c.new_k, c.k_scale), (v, c.new_v, c.v_scale)):
                want = (x.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                nan = torch.isnan(x)
                assert ((got & 0x7f) == 0x7f)[nan].all()
                assert torch.equal(got[~nan], want[~nan]), row.tolist()
