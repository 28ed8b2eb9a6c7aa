"""The first calls of a process, made by several host threads at once (ctypes lets go of the
interpreter's lock inside the library)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import sys, threading
import torch
import gated_delta_rule_153_b200 as gdn
sys.setswitchinterval(1e-6)
gen = torch.Generator(device="cuda").manual_seed(1)
q, k, v = (torch.randn(1, 200, 2, 64, generator=gen, device="cuda").bfloat16() for _ in range(3))
g = -torch.rand(1, 200, 2, generator=gen, device="cuda")
gdn.lib()
ws = [torch.empty(1 << 20, dtype=torch.uint8, device="cuda") for _ in range(16)]
o = [torch.zeros_like(v) for _ in ws]
torch.cuda.synchronize()
gate, errors = threading.Barrier(len(ws)), []
def call(i):
    gate.wait()
    try:
        gdn.gdn_decay_fwd(q, k, v, g, o=o[i], workspace=ws[i], output_final_state=False)
    except Exception as e:
        errors.append(repr(e))
threads = [threading.Thread(target=call, args=(i,)) for i in range(len(ws))]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert not errors, errors
assert all(torch.equal(x, o[0]) for x in o) and o[0].abs().sum() > 0
"""


def test_first_calls_at_once(dev):
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-600:]
