"""CPU: what importing the binding needs, and what its native calls need."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_the_binding_works_without_torch():
    """torch and the module of the native calls are loaded by the calls that use them, not by the import."""
    r = python("""
import sys
sys.modules["torch"] = None      # an import of it raises
from streaming_speaker_diarization_b200 import binding as b
assert b.default_config().n_mels == 128 and b.attn_params(8, 8, 64).scale == 0.125
assert {"sf_kv_append", "sf_encode"} <= set(dir(b)) and not hasattr(b, "sf_nothing")
try:
    b.sf_kv_append
except ImportError as e:
    assert "torch" in str(e), e
else:
    raise SystemExit("loaded")
""")
    assert r.returncode == 0, r.stderr


def test_a_module_that_is_missing_and_one_that_does_not_load_are_told_apart():
    r = python("""
import os
from streaming_speaker_diarization_b200 import binding as b
assert callable(b.sf_attention_packed) and b.sf_attention_packed is b.sf_attention_packed
real = os.path.exists
os.path.exists = lambda p: not str(p).endswith("_calls.so") and real(p)
try:
    b._load_native()
except ImportError as e:
    assert "not built" in str(e), e
else:
    raise SystemExit("loaded")
""")
    assert r.returncode == 0, r.stderr
    r = python("""
import sys
sys.modules["streaming_speaker_diarization_b200._calls"] = None
from streaming_speaker_diarization_b200 import binding as b
try:
    b.sf_attention_packed
except ImportError as e:
    assert "not built" not in str(e), e
else:
    raise SystemExit("loaded")
""")
    assert r.returncode == 0, r.stderr
