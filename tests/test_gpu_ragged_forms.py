"""The forms of the ragged decode (16, 32 and up to 128 rows a key/value head) on the same rows:
each against the definition, and against one another within the sum of their bounds."""
import numpy as np
import pytest
import torch

from bounds import DT, check, f64, half_step
from oracle import operators as ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("few,more", [(16, 17), (32, 33), (32, 128)])
@pytest.mark.parametrize("softcap", [0.0, 8.0])
@pytest.mark.parametrize("alibi,window", [(False, 0), (True, 150)])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_same_rows_in_two_forms(fa, few, more, softcap, alibi, window, d, dtype):
    lens, bs = [1, 200, 1300, 128, 0], 32
    g = torch.Generator().manual_seed(more)
    q = 2 * torch.randn(len(lens), more, 1, d, generator=g).to(DT[dtype])
    kc, vc = torch.randn(2, 5 * 41, 1, bs, d, generator=g).to(DT[dtype])
    table = torch.randperm(5 * 41, generator=g).to(torch.int32).view(5, 41)
    slopes = torch.tensor([2.0 ** -(1 + h % 8) for h in range(more)]) if alibi else None
    got = []
    for n in (few, more):
        s = None if slopes is None else slopes[:n].contiguous()
        x = [q[:, :n].contiguous(), kc, vc, table, torch.tensor(lens, dtype=torch.int32)]
        out, lse = fa.decode_forward_ragged(*(t.to(DEV) for t in x), window=window, softcap=softcap,
                                            slopes=None if s is None else s.to(DEV))
        torch.cuda.synchronize()
        want = ops.ragged_attention(f64(x[0]), f64(kc), f64(vc), table.numpy(), lens, d ** -0.5,
                                    window, softcap, None if s is None else s.numpy(),
                                    half_step(q.dtype))
        check("out", out, want["out"], want["out_tol"])
        check("lse", lse, want["lse"], want["lse_tol"])
        got.append((out[:, :few], lse[:, :few], want))
    want = got[0][2]
    check("out", got[1][0], f64(got[0][0]), 2 * want["out_tol"])
    check("lse", got[1][1], f64(got[0][1]), 2 * want["lse_tol"])
