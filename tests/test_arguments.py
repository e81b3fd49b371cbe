"""Refusals of the binding's argument checks, decided on the host before any launch."""

import os
import sysconfig

import pytest
import torch

from paged_kv_cache_append_gb300 import build, nk
from tests.test_oracle_serving import F32, I32, Fake, _args_append, lib  # noqa: F401


class Scratch(Fake):
    """A workspace as far as the checks look."""

    def element_size(self):
        return self.dtype.itemsize


def shared(*ws, **kw):
    d = dict(pool=0, layer=0, scale=0.1)
    d.update(kw)
    return nk._args().shared_decode(d["pool"], 64, 3, 5, d["layer"], Fake(2, 1, 8, 64), Fake(3, 5, dtype=I32),
                                    Fake(2, dtype=I32), Fake(2, dtype=I32), Fake(1, dtype=I32), d["scale"],
                                    Fake(2, 1, 8, 64), Fake(2, 1, 8, dtype=F32), -1, *ws, 0, 0)


U8 = torch.uint8


@pytest.mark.parametrize("bad", [
    Scratch(4096, dtype=U8, device=-1), Scratch(4096, dtype=U8, device=1), Scratch(4096, dtype=U8, stride=(0,)),
    Scratch(4096, dtype=U8, stride=(2,)), Scratch(64, 64, dtype=F32, stride=(1, 64)),
    Scratch(2, 64, dtype=U8, stride=(0, 1))])
def test_workspace_is_checked(lib, bad):  # noqa: F811
    assert shared(Scratch(4096, dtype=U8)) == -1        # reaches the library, which refuses the NULL pool
    assert shared(Scratch(64, 64, dtype=F32)) == -1
    assert shared(64, 4096) == -1                       # an address and its bytes
    with pytest.raises(ValueError, match="workspace"):
        shared(bad)


def test_shared_decode_refuses_a_host_workspace(lib, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(nk, "_current_stream", lambda dev: 0)
    p = nk.Pool.__new__(nk.Pool)
    p.handle, p.D, p.C, p.L, p.device = 0, 64, 3, 5, 0
    args = (0, Fake(2, 1, 8, 64), Fake(3, 5, dtype=I32), Fake(2, dtype=I32), Fake(2, dtype=I32), Fake(1, dtype=I32), 0.1,
            Fake(2, 1, 8, 64), Fake(2, 1, 8, dtype=F32))
    with pytest.raises(nk.NkError, match="null"):
        p.shared_decode(*args, workspace=Scratch(4096, dtype=U8))
    for bad in (torch.empty(4096, dtype=U8), torch.empty(1, dtype=U8).expand(4096)):
        with pytest.raises(ValueError, match="workspace"):
            p.shared_decode(*args, workspace=bad)


def test_the_argument_module_is_named_for_its_interpreter(lib):  # noqa: F811
    """Built against one version's headers: another version must not find it,
    nor one without a tag, which every version would load."""
    untagged = os.path.join(nk.PKG, "_pyargs.so")
    with open(untagged, "wb"):
        pass
    try:
        path = build.build_pyargs()
        assert os.path.basename(path) == "_pyargs" + sysconfig.get_config_var("EXT_SUFFIX")
        assert not os.path.exists(untagged)
        assert nk._args().__file__ == path
    finally:
        if os.path.exists(untagged):
            os.remove(untagged)


@pytest.mark.parametrize("layer,error", [(None, TypeError), ("0", TypeError), (1.5, TypeError), (1 << 70, OverflowError)])
def test_a_layer_that_is_no_number_is_named(lib, layer, error):  # noqa: F811
    """The error that the number raises, not one of the calls that follow."""
    assert shared(64, 4096, layer=0) == -1 and _args_append(layer=0) == -1
    with pytest.raises(error):
        shared(64, 4096, layer=layer)
    with pytest.raises(error):
        _args_append(layer=layer)
