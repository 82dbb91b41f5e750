"""A gradient group's tables against its tensors. On the host: the extension sees a tensor whose storage, size, type or
layout is not the tabulated one any more. On the GPU: calls follow tensors whose storage was replaced."""
import ctypes
import math

import pytest
import torch

import resharding_tensor_parallelism_gb300 as rtp
from resharding_tensor_parallelism_gb300 import _build

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def _tables(ts):
    arrays = (rtp._i32([rtp._dtype_code(t) for t in ts]), rtp._i64([t.numel() for t in ts]),
              rtp._ptrs([t.data_ptr() for t in ts]))
    return arrays, [ctypes.addressof(a) for a in arrays]


CHANGES = {
    "storage": lambda ts: setattr(ts[0], "data", ts[0].clone()),
    "set_": lambda ts: ts[1].set_(torch.zeros(7)),
    "size": lambda ts: setattr(ts[0], "data", ts[0][:9].clone()),
    "view of it": lambda ts: setattr(ts[0], "data", ts[0][1:]),
    "type": lambda ts: ts.__setitem__(1, ts[1].to(BF16)),
    "layout": lambda ts: setattr(ts[2], "data", ts[2].t()),
    "another tensor": lambda ts: ts.__setitem__(0, ts[0].clone()),
    "no tensor": lambda ts: ts.__setitem__(0, None),
    "fewer": lambda ts: ts.pop(),
    "more": lambda ts: ts.append(torch.zeros(3)),
}


@pytest.mark.parametrize("change", CHANGES)
def test_the_extension_sees_what_changed(change):
    ext = rtp._tables()
    ts = [torch.zeros(10, dtype=BF16), torch.zeros(7), torch.zeros(3, 4), torch.zeros(0)]
    arrays, at = _tables(ts)
    keep = list(ts), [t.detach() for t in ts]  # no storage is freed
    args = lambda: (len(arrays[1]), *at, ts, -1)  # host tensors are on "device" -1
    assert ext.unchanged(*args()) is True
    for t in ts:
        t.add_(1)
    assert ext.unchanged(*args()) is True  # new values are no change
    CHANGES[change](ts)
    assert ext.unchanged(*args()) is False
    # the whole call hands such a group back before it calls the library
    assert ext.clip(len(arrays[1]), *at, 0, 0, 1.0, None, ts, -1, 0) is None
    del keep


def test_unchanged_refuses_wrong_arguments():
    for args in ((), (1, 2, 3, 4, (), 0), ("n", 0, 0, 0, [], 0)):
        with pytest.raises(TypeError):
            rtp._tables().unchanged(*args)


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["clip", "clip out", "clip stream", "norm"])
def test_replaced_storage_is_followed(how):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rand = lambda n, dtype: (torch.randn(n, generator=gen, device="cuda") * 1e-2).to(dtype)
    grads = [rand(5000, BF16), rand(70000, F32), rand(33, F32)]
    group = rtp.GradGroup(grads)
    group.norm()
    for change in (lambda: setattr(grads[0], "data", rand(5000, BF16)), lambda: grads[1].set_(rand(90001, F32)),
                   lambda: setattr(grads[2], "data", rand(8, F32))):
        old = [t.detach() for t in grads]  # the storage before, and what it holds
        change()
        held = [t.clone() for t in old]
        before = [t.clone() for t in grads]
        want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))
        torch.cuda.synchronize()
        if how == "norm":
            assert abs(float(group.norm()) - want) <= 2.0 ** -17 * want  # bound: test_gpu_grad_norm.py
            continue
        out = [torch.empty_like(t) for t in grads] if how == "clip out" else None
        norm, got = group.clip(0.05, out=out, stream=torch.cuda.current_stream() if how == "clip stream" else None)
        assert abs(float(norm) - want) <= 2.0 ** -17 * want
        c = min(1.0, 0.05 / (want + 1e-6))
        for t, b, o, h, g in zip(got, before, old, held, grads):
            ref = b.double() * c
            assert bool(((t.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -16) * ref.abs()).all())
            if o.data_ptr() != g.data_ptr():
                assert torch.equal(o, h)  # the storage that the tensor left is not written
    assert rtp.device_error() == 0


@pytest.mark.gpu
def test_changed_groups_that_are_refused():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    for change, error in ((lambda ts: setattr(ts[0], "data", ts[0].t()), rtp.RtpError),
                          (lambda ts: setattr(ts[0], "data", ts[0].cpu()), rtp.RtpError), (lambda ts: ts.pop(), rtp.RtpError),
                          (lambda ts: ts.__setitem__(1, ts[1].double()), TypeError)):
        group = rtp.GradGroup([torch.ones(5, 8, device="cuda"), torch.ones(9, device="cuda")])
        change(group.grads)
        for call in (group.norm, lambda: group.clip(1.0)):
            with pytest.raises(error):
                call()


@pytest.mark.gpu
def test_the_result_is_the_callers_list():
    """What a caller does with the list that clip returns does not change the group, nor does the list given to it."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    grads = [torch.ones(5, device="cuda"), torch.ones(9, device="cuda")]
    group = rtp.GradGroup(grads)
    for kw in ({}, {"stream": torch.cuda.current_stream()}):
        _, got = group.clip(1e9, **kw)
        assert type(got) is list and all(a is b for a, b in zip(got, grads))
        got.pop()
    grads.pop()
    assert abs(float(group.norm()) - 14 ** 0.5) <= 2.0 ** -17 * 14 ** 0.5
    out = [torch.empty(5, device="cuda"), torch.empty(9, device="cuda")]
    assert group.clip(1e9, out=out)[1] is out
