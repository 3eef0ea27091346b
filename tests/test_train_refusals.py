"""Calls out of order: refused on the host (no GPU needed; nothing is launched)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _layer(**kw):
    from combine_top_router_amd import lib as L
    if not os.path.exists(L.lib_path()):
        pytest.skip("libmoe.so not built")
    from combine_top_router_amd import MoeLayer
    return MoeLayer(16, 64, 64, 8, 2, device="cpu", **kw)


@pytest.mark.parametrize("recompute", [0, 1])
def test_updates_need_gradients(recompute):
    """The gradients' buffers hold whatever was in the memory until a backward has run."""
    lay = _layer(recompute=recompute)
    with pytest.raises(RuntimeError, match="without a backward"):
        lay.orthogonalize()
    assert not lay._updates and not lay._orth   # nothing allocated either


def test_a_balance_loss_needs_a_forward():
    with pytest.raises(RuntimeError, match="without a forward"):
        _layer().balance(0.1)


def test_imports_without_torchs_private_names():
    """A torch without them (built for the CPU) imports the classes, and has the public calls."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "from combine_top_router_amd import layer\n"
            "torch.cuda.current_device = lambda: 3\n"
            "class S: cuda_stream = 7\n"
            "torch.cuda.current_stream = lambda index: S\n"
            "assert layer._current_device() == 3 and layer._raw_stream(0) == 7\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.stderr
