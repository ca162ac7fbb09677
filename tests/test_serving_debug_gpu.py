"""The serving operators through the debug build (libaxr_debug.so): every plain load and
store stays inside the buffers that the call describes.  Run in processes of their own,
as the library is chosen once per process: the operators' own tests, which require
device status 0, and this file as a script, where every span is 4 bytes short and each
call must record status bit 16 and leave the last bytes of its outputs as they were."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
sys.path[:0] = [p for p in (HERE, ROOT) if p not in sys.path]
pytestmark = pytest.mark.gpu


def _run(args):
    from lut_attention_b200 import build

    if not os.path.exists(build.DEBUG_LIB_PATH):
        build.build(debug=True)
    r = subprocess.run([sys.executable, *args], cwd=ROOT, env=dict(os.environ, AXR_DEBUG="1"), capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    return r.stdout


def test_operators_stay_inside_their_buffers():
    out = _run(["-m", "pytest", os.path.join(HERE, "test_serving_gpu.py"), "-q", "-m", "gpu", "-x", "-k",
                "types_and or lengths or widths or masked or larger or leaves or ignores"])
    assert "passed" in out and "failed" not in out


def test_checks_fire_on_shortened_spans():
    assert "4 calls recorded" in _run([os.path.abspath(__file__)])


def _slack():
    import torch

    from lut_attention_b200 import axr, workloads

    assert axr.axr_debug_build()
    axr.axr_debug_set_span_slack(4)
    dev, calls = "cuda", 0

    def recorded(what):
        nonlocal calls
        torch.cuda.synchronize()
        assert axr.axr_device_status() & 16, what
        calls += 1

    x = torch.randn((2, 40, 32), device=dev)
    out, lse = torch.full_like(x, 7.0), torch.full((2, 40), 7.0, device=dev)
    axr.axr_prompt_attention(x, x, x, torch.tensor([0, 40], dtype=torch.int32, device=dev), out=out, lse=lse)
    recorded("prompt")
    assert out.view(-1)[-1] == 7.0 and lse.view(-1)[-1] == 7.0
    idx, norms = workloads.make_random_packed(2, 40, 64, 4, seed=1, device=dev)
    V = torch.randn((2, 40, 64), device=dev).to(torch.bfloat16)
    signs = torch.ones(64, dtype=torch.int8, device=dev)
    out, lse = torch.full((4, 64), 7.0, dtype=torch.bfloat16, device=dev), torch.full((4,), 7.0, device=dev)
    axr.axr_attention_shared(torch.randn((4, 64), device=dev), idx, norms, V, idx, norms, V,
                             torch.tensor([40], dtype=torch.int32, device=dev), 2, 4, signs, out=out, lse=lse)
    recorded("shared")
    assert out.view(-1)[-1] == 7.0 and lse[-1] == 7.0
    sums = torch.full((2, 40), 7.0, device=dev)
    axr.axr_accumulate_weights(torch.randn((4, 40), device=dev), sums, 2)
    recorded("weights")
    assert sums[-1, -1] == 7.0
    got = (torch.full((2, 30, 32), 77, dtype=torch.uint8, device=dev), torch.full((2, 30), 7.0, device=dev),
           torch.full((2, 30, 64), 7.0, dtype=torch.bfloat16, device=dev), torch.full((2, 30), 7.0, device=dev),
           torch.full((2, 30), -9, dtype=torch.int32, device=dev), torch.full((2,), -9, dtype=torch.int32, device=dev))
    axr.axr_evict(idx, norms, V, torch.rand((2, 40), device=dev),
                  torch.tensor([40, 40], dtype=torch.int32, device=dev), 30, 4, out=got)
    recorded("evict")
    assert got[0].view(-1)[-1] == 77 and got[2].view(-1)[-1] == 7.0 and got[4][-1, -1] == -9 and got[5][-1] == -9
    print(f"{calls} calls recorded")


if __name__ == "__main__":
    _slack()
