"""The binding where torch lacks the 8-bit exponents' type: it imports, and only their calls are refused."""

import os
import subprocess
import sys

CODE = """
import torch
del torch.float8_e8m0fnu
import sparse_attention_kv_dsa_gb300.echo as E
assert E.paged_decode_workspace_bytes(8, 2, 64) > 0
codes = torch.zeros(1, 8, 2, 64, dtype=torch.uint8)
for call in (lambda: E._scales(codes[..., 0], codes[..., 0], codes, "call"), lambda: E._scales(None, None, codes, "call")):
    try:
        call()
        raise SystemExit("scales were taken")
    except E.EchoError as e:
        assert e.code == E.ERR_INVALID_ARG
"""


def test_a_torch_without_the_exponents_type():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
