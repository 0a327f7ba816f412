"""Without the built library every call raises, at once."""
import subprocess
import sys

from mla_causal_attention_gb300.build import ROOT


def test_missing_library_raises():
    code = ("from mla_causal_attention_gb300 import binding\n"
            "binding.LIB_PATH += '.none'\n"
            "try:\n"
            "    binding.mla_attn_workspace_bytes(1, 1, 1, 1)\n"
            "except binding.MlaAttnError as e:\n"
            "    print('raised', e.status.name, 'is not built' in str(e))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=120)
    assert r.stdout.strip() == "raised ERR_CUDA True", r.stdout + r.stderr
