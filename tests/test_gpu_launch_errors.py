"""A launch that fails is reported under the entry point's own name.

The launches go to a stream whose capture has been given up (a synchronisation
inside it ends it with an error): the runtime refuses them, nothing runs.  In a
process of its own, since the capture's allocations are lost with it.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import torch
import block_quantized_moe_layer_gb300 as pkg

i32 = dict(dtype=torch.int32, device="cuda")
starts, lens, table = torch.tensor([0, 40], **i32), torch.tensor([50], **i32), torch.arange(4, **i32)[None]
parents, path = torch.arange(-1, 39, **i32), torch.arange(40, **i32)[None]
calls = {}
for act, dt in ((pkg.ACT_BF16, torch.bfloat16), (pkg.ACT_F32, torch.float32)):
    for hq in (1, 4, 16):
        at = pkg.Attention(hq, 1, 64, 16, 4, 40, 1, 64, rot_dim=0, act=act)
        q, pages, out, new = torch.zeros(40, hq, 64, device="cuda", dtype=dt), at.pages("cuda"), torch.empty(40, hq, 64, device="cuda", dtype=dt), torch.empty(1, **i32)
        for n in (1, 40):
            one = (q[:n], pages, torch.tensor([0, n], **i32), lens, table, n, 50)
            calls[f"moe_attn_forward {act} {hq} {n}"] = lambda st, at=at, one=one, o=out[:n]: at.forward(*one, out=o, stream=st)
            calls[f"moe_attn_forward_tree {act} {hq} {n}"] = lambda st, at=at, one=one, o=out[:n], p=parents[:n]: at.forward(*one, out=o, stream=st, parents=p)
    calls[f"moe_attn_commit {act}"] = lambda st, at=at, pages=pages, new=new: at.commit(pages, starts, lens, table, path, 50, new_lens=new, stream=st)
for call in calls.values():
    call(torch.cuda.current_stream())
torch.cuda.synchronize()
st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.stream(st):
    g.capture_begin(capture_error_mode="relaxed")
    try:
        st.synchronize()
        raise SystemExit("a synchronisation was captured")
    except RuntimeError:
        pass
    for name, call in calls.items():
        try:
            call(st)
        except pkg.MoEError as e:
            assert name.split()[0] + " launch" in str(e), (name, str(e))
        else:
            raise SystemExit(f"{name}: a launch into a capture that is lost")
print("named", len(calls))
"""


def test_failed_launches_name_their_entry_point():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE], cwd=root, capture_output=True, text=True, timeout=300)
    assert "named" in r.stdout, r.stdout + r.stderr
