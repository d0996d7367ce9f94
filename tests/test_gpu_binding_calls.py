"""What a call through the Python binding does beside the computation: other threads run while it
allocates and launches, and a call that is refused has changed nothing."""
import ctypes
import shutil
import subprocess
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# A stand-in for the library whose every call waits (5 s at most) until the test lets it go on,
# as a launch waits for room in a full queue. It makes no GPU call.
FAKE = """
#include <unistd.h>
volatile int entered, go;
static int hold(void) {
  int i;
  entered = 1;
  for (i = 0; i < 500 && !go; ++i) usleep(10000);
  i = go ? -100 : -200;
  entered = go = 0;
  return i;
}
int fa_fwd_span(void) { return hold(); }
int fa_bwd_span(void) { return hold(); }
int fa_fwd_ragged_paged(void) { return hold(); }
int fa_qk_norm_rope(void) { return hold(); }
int fa_qk_norm_rope_bwd(void) { return hold(); }
int fa_qk_norm_rope_append(void) { return hold(); }
unsigned long fa_bwd_span_workspace_bytes(void) { return 256; }
unsigned long fa_fwd_ragged_paged_workspace_bytes(void) { return 256; }
unsigned long fa_qk_norm_rope_bwd_workspace_bytes(void) { return 256; }
"""


@pytest.fixture(scope="module")
def waiting_library(tmp_path_factory):
    cc = shutil.which("gcc") or shutil.which("cc") or shutil.which("g++")
    at = tmp_path_factory.mktemp("fake")
    (at / "fake.c").write_text(FAKE)
    subprocess.run([cc, "-x", "c", "-O1", "-shared", "-fPIC", str(at / "fake.c"), "-o",
                    str(at / "fake.so")], check=True)
    return ctypes.CDLL(str(at / "fake.so"))


@pytest.mark.parametrize("name", ["span_forward", "span_backward", "ragged", "norm_rope",
                                  "norm_rope_bwd", "append", "step"])
def test_other_threads_run_while_a_call_waits(fa, waiting_library, name):
    L = waiting_library
    h = L._handle
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device=DEV)
    i = torch.zeros(1, 4, dtype=torch.int32, device=DEV)
    lse = torch.zeros(1, 2, 4, device=DEV)
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    n, table = i[0, :1].contiguous(), i[:, :2].contiguous()
    args = dict(
        span_forward=(h, q, q, q, i, i, None, None, 0.0, None, None, None),
        span_backward=(h, q, q, q, i, i, q, q, lse, None, None, None, None, 0.0, None, None, None),
        ragged=(h, q, kc, kc, table, n, None, None, None, 0, 0.0, None, None, None),
        norm_rope=(h, q, q, None, None, None, None, None, None, 1e-6, False, 1.0, None),
        norm_rope_bwd=(h, q, q, q, q, None, None, None, None, None, None, None, None, None, 1e-6,
                       False, 1.0, True, None),
        append=(h, q, q, q, None, kc, kc, table, n, None, None, None, 1e-6, False, 1.0, None),
        step=(h, q, q, q, kc, kc, table, n, None, None, None, 1e-6, False, 1.0, 0, 0.0, None, None,
              None))[name]
    call = getattr(fa._native(), name)
    entered, go = (ctypes.c_int.in_dll(L, s) for s in ("entered", "go"))
    got, entered.value, go.value = [], 0, 0
    t = threading.Thread(target=lambda: got.append(call(*args)))
    t.start()
    while not entered.value and t.is_alive():
        pass
    go.value = 1          # reached while the call waits only if the call let this thread run
    t.join()
    assert got == [-100]


def step_args(B=2, Hq=4, Hkv=2, Sq=1, d=64, dtype=torch.bfloat16, bs=16, mb=4):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)
    kc, vc = r(B * mb, Hkv, bs, d), r(B * mb, Hkv, bs, d)
    table = torch.arange(B * mb, dtype=torch.int32, device=DEV).view(B, mb)
    lens = torch.full((B,), Sq + 3, dtype=torch.int32, device=DEV)
    turns = torch.zeros(d // 2, dtype=torch.int64, device=DEV)
    return [r(B, Hq, Sq, d), r(B, Hkv, Sq, d), r(B, Hkv, Sq, d), kc, vc, table, lens, turns]


@pytest.mark.parametrize("sizes,kw", [
    (dict(Hq=32, Hkv=1, Sq=5), dict()),                # 160 rows a key/value head
    (dict(dtype=torch.float32), dict()),
    (dict(), dict(window=-1)), (dict(), dict(softcap=-1.0)), (dict(), dict(softcap=float("nan"))),
    (dict(), dict(scale=0.0)), (dict(), dict(slopes="short")), (dict(), dict(window="text")),
    (dict(), dict(eps=-1.0, weights=True)), (dict(), dict(rope_scale=float("inf"))),
])
def test_a_refused_step_leaves_the_cache_alone(fa, sizes, kw):
    a = step_args(**sizes)
    kc, vc = a[3].clone(), a[4].clone()
    kw = dict(kw)
    if kw.get("slopes") == "short":
        kw["slopes"] = torch.ones(3, device=DEV)
    if kw.pop("weights", False):
        kw["q_weight"] = kw["k_weight"] = torch.ones(64, dtype=a[0].dtype, device=DEV)
    with pytest.raises((fa.FAError, ValueError, TypeError)):
        fa.decode_step_ragged(*a, **kw)
    torch.cuda.synchronize()
    assert torch.equal(a[3], kc) and torch.equal(a[4], vc)


def test_a_step_is_its_two_calls(fa):
    a = step_args(Sq=3)
    b = [t.clone() for t in a]
    out, lse = fa.decode_step_ragged(*a, window=3, softcap=9.0)
    q = fa.qk_norm_rope_append(*b)
    want = fa.decode_forward_ragged(q, *b[3:7], window=3, softcap=9.0)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(a[3], b[3]) and torch.equal(a[4], b[4])
