"""NaN and infinity where a row of the ragged paged decode sees them: out and lse both say so,
in one share or joined from several, and every other row stays within its bound."""
import numpy as np
import pytest
import torch

from bounds import DT, check, f64, half_step
from oracle import operators as ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LENS, BS = [700, 5000, 3, 0], 64
FORMS = [(8, 2), (24, 1), (40, 1), (128, 1)]   # 4, 24, 40 and 128 rows a key/value head


def make(Hq, Hkv, d, dtype):
    g = torch.Generator().manual_seed(Hq + d)
    per = -(-max(LENS) // BS)
    nb = len(LENS) * per
    q = torch.randn(len(LENS), Hq, 1, d, generator=g).to(DT[dtype])
    kc, vc = torch.randn(2, nb, Hkv, BS, d, generator=g).to(DT[dtype])
    table = torch.randperm(nb, generator=g).to(torch.int32).view(len(LENS), per)
    return [q, kc, vc, table, torch.tensor(LENS, dtype=torch.int32)]


def run(fa, x, **kw):
    out, lse = fa.decode_forward_ragged(*(t.to(DEV) for t in x), **kw)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0
    return out.cpu(), lse.cpu()


def compare_rest(got, clean, bad, softcap):
    """Rows that see no NaN, against the definition on inputs without it."""
    q, kc, vc, table, lens = clean
    want = ops.ragged_attention(f64(q), f64(kc), f64(vc), table.numpy(), lens.tolist(),
                                q.shape[-1] ** -0.5, 0, softcap, u=half_step(q.dtype))
    bad = bad.numpy()
    for name, t in zip(("out", "lse"), got):
        check(name, f64(t)[~bad], want[name][~bad], want[name + "_tol"][~bad])


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("Hq,Hkv", FORMS)
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_nan_in_one_query(fa, Hq, Hkv, d, dtype, softcap):
    x = make(Hq, Hkv, d, dtype)
    y = [t.clone() for t in x]
    bad = torch.zeros(len(LENS), Hq, 1, dtype=torch.bool)
    for b, h in ((0, Hq - 1), (1, 5)):
        y[0][b, h, 0, 9] = float("nan")
        bad[b, h] = True
    got = run(fa, y, softcap=softcap)
    assert torch.equal(got[1].isnan(), bad) and torch.equal(got[0].isnan().all(-1), bad)
    compare_rest(got, x, bad, softcap)


@pytest.mark.parametrize("at", [0, 4321, 4999])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("Hq,Hkv", FORMS)
def test_nan_in_a_key_that_is_seen(fa, Hq, Hkv, at, softcap):
    x = make(Hq, Hkv, 128, "bf16")
    y = [t.clone() for t in x]
    y[1][y[3][1, at // BS], 0, at % BS, 3] = float("nan")
    bad = torch.zeros(len(LENS), Hq, 1, dtype=torch.bool)
    bad[1, :Hq // Hkv] = True
    got = run(fa, y, softcap=softcap)
    assert torch.equal(got[1].isnan(), bad) and torch.equal(got[0].isnan().all(-1), bad)
    compare_rest(got, x, bad, softcap)


@pytest.mark.parametrize("Hq,Hkv", FORMS)
def test_infinite_scores(fa, Hq, Hkv):
    """+infinity among a row's scores leaves no weights: NaN, in lse too. A score of -infinity has
    weight 0, and a row of none but such scores is like one that sees nothing."""
    x = make(Hq, Hkv, 64, "bf16")
    x[0][:, :, 0, 4] = 1.0
    x[0][1, 0, 0, 4] = -1.0                          # this row's score is -infinity: weight 0
    x[1][x[3][1, 40], 0, 7, 4] = float("inf")
    x[4][0] = 1
    x[1][x[3][0, 0], 0, 0, 4] = float("-inf")
    out, lse = run(fa, x)
    G = Hq // Hkv
    assert out[1, 1:G].isnan().all() and lse[1, 1:G].isnan().all()
    assert out[1, 0].isfinite().all() and lse[1, 0].isfinite().all()
    assert (out[0, :G] == 0).all() and (lse[0, :G] == float("-inf")).all()
    assert (out[3] == 0).all() and (lse[3] == float("-inf")).all()      # no keys
