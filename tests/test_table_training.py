"""A tensor that the binding's extension cannot take an address of raises from the loss calls and the AdamW step too; it
does not end the process. No GPU needed: a tensor wrapped by torch.func over one that only says it is on a GPU."""
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
def t(*shape, dtype=b):
    return torch.empty(shape, dtype=dtype, device="cuda:0")
W, y = [t(16, 8), t(16, 8)], t(4, dtype=torch.int64)
table = (rtp.AdamWTensor * 1)()
table[0].numel, table[0].param_dtype = 16, 1
import ctypes
at = ctypes.addressof(table)
def wrapped(call, arg):
    try:
        got = torch.func.vmap(call)(arg)
    except RuntimeError as e:
        print("raised:", str(e).splitlines()[0][:200])
    else:
        print("returned:", got)
"""

CALLS = {
    "loss, X": "wrapped(lambda x: ext.loss(x, W, y, -1, -100, 0, 0), t(3, 4, 16))",
    "loss, W": "wrapped(lambda w: ext.loss(t(4, 16), [w, w], y, -1, -100, 0, 0), t(3, 16, 8))",
    "loss, targets": "wrapped(lambda v: ext.loss(t(4, 16), W, v, -1, -100, 0, 0), t(3, 4, dtype=torch.int64))",
    "loss_train, X": "wrapped(lambda x: ext.loss_train(x, W, y, None, -1, -100, True, 1.0, 0, 0), t(3, 4, 16))",
    "adamw, params": "wrapped(lambda p: ext.adamw(at, 1, [p], [None], [t(16)], 32, 0.1, 1e-8, None, 1.0, 0, 4096, 0, 0), t(3, 16))",
    "adamw, grads": "wrapped(lambda g: ext.adamw(at, 1, [t(16)], [None], [g], 32, 0.1, 1e-8, None, 1.0, 0, 4096, 0, 0), t(3, 16))",
    "adamw, norm": "wrapped(lambda v: ext.adamw(at, 1, [t(16)], [None], [t(16)], 32, 0.1, 1e-8, v, 1.0, 0, 4096, 0, 0),"
                   " t(3, 1, dtype=torch.float32))",
}


@pytest.mark.parametrize("name", CALLS)
def test_a_tensor_without_storage(name):
    _build.build()
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", SETUP + CALLS[name]], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert r.stdout.startswith("raised:") and "storage" in r.stdout.lower(), r.stdout


def test_a_list_of_another_length_than_the_groups_table():
    """The extension hands such a call back: it neither reads nor writes behind the table."""
    _build.build()
    code = SETUP + """
rows = (rtp.AdamWTensor * 3)()
for r in rows:
    r.numel, r.param_dtype, r.param = 16, 1, 4096
at = ctypes.addressof(rows)
for n, lists in ((1, ([t(16), t(16)], [None, None], [t(16), t(16)])), (1, ([t(16)], [None], [])), (1, ([t(16)], [], [t(16)])),
                 (1, ([], [None], [t(16)]))):
    assert ext.adamw(at, n, *lists, 32, 0.1, 1e-8, None, 1.0, 0, 4096, 0, 0) is None, (n, lists)
assert all(r.param == 4096 and not r.grad for r in rows)
print("handed back")
"""
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "handed back\n", (r.returncode, r.stdout, r.stderr[-500:])


def test_the_binding_passes_the_tables_own_length(monkeypatch):
    """Lists that grew after the group was built do not make a step reach behind its table. No GPU: the call is recorded."""
    import torch

    import resharding_tensor_parallelism_gb300 as rtp
    asked = []

    class Extension:
        @staticmethod
        def adamw(table, n, *rest):
            asked.append(n)

    group = object.__new__(rtp.AdamWGroup)
    group.params, group.masters = [torch.zeros(4), torch.zeros(4)], [None, None]
    group.states, group.lr, group.eps, group.seed, group._index, group._clock_at = 32, 0.1, 1e-8, 0, 0, 4096
    group._table = (rtp.AdamWTensor * 1)()
    group._table_at, group._numels = 4096, [4]
    monkeypatch.setattr(rtp, "_ext", Extension)
    monkeypatch.setattr(rtp.AdamWGroup, "_begin", lambda self, stream: 0)
    for grads in ([torch.zeros(4)] * 2, [torch.zeros(4)]):
        with pytest.raises(rtp.RtpError):
            group.step(grads)
    assert asked == [1, 1]
