"""The sign of zeros in e4m3 rows: -0 / scale is -0, and a negative value too small for e4m3
rounds to -0, at every scale."""

import numpy as np
import pytest
import torch

import unpermute_ffnwb_batching_amd as F
from oracle import expert_ffn as O

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_zeros_keep_their_sign(dtype):
    # rows whose scales lie in the middle of the range and, in 32 bits, past both of its ends, where the
    # quotients come from divisions
    g = torch.Generator().manual_seed(301)
    sizes = [1.0, 2.0 ** -6, 3000.0] + ([2.0 ** -100, 2.0 ** 120] if dtype == torch.float32 else [])
    x = torch.randn((len(sizes) + 1, 300), generator=g) * torch.tensor(sizes + [0.0])[:, None]
    x[:, ::3] = 0.0
    x[:, 1::3] = -0.0
    x[:, 5] = -x[:, 2].abs() * 1e-6     # rounds to -0
    x = x.to(dtype)
    print(f"quant: signed zeros {dtype}", flush=True)
    out = F.moe_quant_fp8(x.cuda())
    torch.cuda.synchronize()
    want, scales = O.quantise_rows(x.float().numpy())
    assert (want[:, 1::3] == 0x80).all() and (want[:, ::3] == 0).all() and (want[:-1, 5] == 0x80).all()
    np.testing.assert_array_equal(out["q"].view(torch.uint8).cpu().numpy(), want)
    np.testing.assert_array_equal(out["scale"].cpu().numpy(), scales)
