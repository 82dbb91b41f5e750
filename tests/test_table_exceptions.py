"""A tensor that the binding's extension cannot take an address of raises; it does not end the process. No GPU needed: a
tensor wrapped by torch.func over one that only says it is on a GPU has no storage. In child processes, since an
exception that leaves the extension ends the interpreter."""
import subprocess
import sys

import pytest

from resharding_tensor_parallelism_gb300 import _build

SETUP = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import resharding_tensor_parallelism_gb300 as rtp
ext = rtp._tables()
b = torch.bfloat16
mode = FakeTensorMode()
mode.__enter__()
def t(*shape):
    return torch.empty(shape, dtype=b, device="cuda:0")
W, R, batch, wide = [t(16, 8), t(16, 8)], t(4, 8), t(3, 4, 16), t(3, 16, 8)
def wrapped(call, arg):
    try:
        got = torch.func.vmap(call)(arg)
    except RuntimeError as e:
        print("raised:", str(e).splitlines()[0][:200])
    else:
        print("returned:", got)
"""

CALLS = {
    "linear, X": "wrapped(lambda x: ext.linear(x, W, False, None, None, 0, 0, 0), batch)",
    "linear, W": "wrapped(lambda w: ext.linear(t(4, 16), [w, w], False, None, None, 0, 0, 0), wide)",
    "linear, bias": "wrapped(lambda v: ext.linear(t(4, 16), W, False, [v, v], None, 0, 0, 0), t(3, 8))",
    "linear, residual": "wrapped(lambda r: ext.linear(t(4, 16), W, False, None, [r, r], 0, 0, 0), t(3, 4, 8))",
    "glu, X": "wrapped(lambda x: ext.glu(x, W, W, [t(8, 16), t(8, 16)], None, 3, 0, 0), batch)",
    "glu, B": "wrapped(lambda v: ext.glu(t(4, 16), W, W, [v, v], None, 3, 0, 0), t(3, 8, 16))",
    "table": "wrapped(lambda x: ext.table([x], (4, 16), 1, 0), batch)",
    "like": "wrapped(lambda x: ext.like([x], [t(4, 16)], 0), batch)",
}


@pytest.mark.parametrize("name", CALLS)
def test_a_tensor_without_storage(name):
    _build.build()
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", SETUP + CALLS[name]], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert r.stdout.startswith("raised:") and "storage" in r.stdout.lower(), r.stdout


def test_the_calls_of_the_binding_raise():
    """grad and vmap of a linear layer or a gated block, through the public calls."""
    _build.build()
    code = SETUP + """
torch._C._cuda_getDevice = lambda: 0
rtp._stream_ptr = lambda stream: None
wrapped(lambda x: rtp.tp_linear(x, W)[0], batch)
wrapped(lambda x: rtp.tp_glu(x, W, W, [t(8, 16), t(8, 16)]), batch)
"""
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.count("raised:") == 2, (r.returncode, r.stdout, r.stderr[-500:])
