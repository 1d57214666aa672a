"""GPU: engines made and destroyed through the library's own functions, in the native calls."""
import ctypes

import pytest

from _helpers import tiny_weights

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
from streaming_speaker_diarization_b200 import binding as b  # noqa: E402
from synth import weights_blob  # noqa: E402


@pytest.mark.parametrize("precision", [0, 1])
def test_an_engine_from_a_file(tmp_path, precision):
    path = tmp_path / "weights"
    path.write_bytes(weights_blob(tiny_weights()))
    h = ctypes.c_void_p()
    cfg = b.default_config(n_conformer=2, n_transformer=2, precision=precision, max_batch=1)
    b._check(b.lib.sf_create_from_file(str(path).encode(), ctypes.byref(cfg), ctypes.byref(h)))
    assert b._engines[h.value] == (precision, torch.cuda.current_device())
    x = torch.randn(3, 2, 64, device="cuda").to(torch.bfloat16 if precision else torch.float32)
    cu, p = torch.tensor([0, 3], dtype=torch.int32, device="cuda"), b.attn_params(2, 2, 64, left=0, right=0)
    for eng in (h.value, h):
        out = torch.zeros_like(x)
        b.sf_attention_packed(eng, x, x, x, cu, out, p)
        b.sf_check(eng)
        assert torch.equal(out, x)
    with pytest.raises(b.SFError, match="SF_EINVAL: k must be"):
        b.sf_attention_packed(h, x, x.double(), x, cu, out, p)
    y = torch.zeros(3, 2, 32, device="cuda", dtype=x.dtype)
    with pytest.raises(b.SFError, match="SF_ESHAPE: head_dim"):   # refused by the library itself
        b.sf_attention_packed(h, y, y, y, cu, y, b.attn_params(2, 2, 32))
    torch.cuda.synchronize()
    b._check(b.lib.sf_destroy(h))
    with pytest.raises(b.SFError, match="not an engine"):
        b.sf_attention_packed(h, x, x, x, cu, out, p)
