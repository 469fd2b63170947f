"""Which GPU a call goes to, without one: tensors that say where they are, a library that
notes what it was given."""
import types

import pytest
import torch

from drift_aware_kv_spherical_gb300 import polestar as ps


class On:
    """What the binding asks of a device tensor."""
    is_cuda = True

    def __init__(self, index, shape, dtype=torch.float32):
        self.index, self.shape, self.dtype = index, torch.Size(shape), dtype
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def stride(self):
        return ()

    def data_ptr(self):
        return 0x1000 * (1 + self.index)


@pytest.fixture
def calls(monkeypatch):
    made = []
    lib = types.SimpleNamespace(
        handle=lambda device=None: ("handle", device),
        cdll=types.SimpleNamespace(ps_commit_drawn=lambda *a: made.append(a) or 0))
    monkeypatch.setattr(ps, "_lib", lambda: lib)
    monkeypatch.setattr(ps, "_raw_stream", lambda index: ("stream", index))
    return made


def _commit(conf, other, role=None):
    u8 = torch.uint8
    ps.ps_commit_drawn(conf, role or On(other, (8,), u8), On(other, (2, 8), u8), On(other, (2, 8)),
                       8, On(other, (2, 8)), On(other, (2, 8), torch.int32), On(other, (2, 8)),
                       None, 8, ps.CommitParams(0.9, 1, 0.1, 0, 1), On(other, (2, 8), u8))


def test_drawn_tokens_are_committed_where_they_are(calls):
    """Not on the current GPU, whose stream and handle are another's."""
    _commit(On(1, (2, 8)), 1)
    (handle, *_, stream), = calls
    assert handle == ("handle", 1) and stream == ("stream", 1)


def test_tensors_of_two_gpus_are_refused(calls):
    with pytest.raises(ValueError, match="GPU 1"):
        _commit(On(1, (2, 8)), 0)
    with pytest.raises(ValueError, match="GPU 1"):
        _commit(On(1, (2, 8)), 1, role=On(0, (8,), torch.uint8))
    with pytest.raises(ValueError):
        _commit(On(1, (2, 8), torch.float64), 1)
    with pytest.raises(ValueError):
        _commit(torch.zeros(2, 8), 1)
    z = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="device tensor"):
        ps.ps_commit_drawn(z, z, z, z, 8, z, z, z, None, 8, ps.CommitParams(0.9, 1, 0.1, 0, 1), z)
    assert not calls
