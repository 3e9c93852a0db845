"""The example's attention layer with head norms and over an 8-bit cache: chunks and decoding agree with the prompt in one
piece over a 16-bit cache as far as the codes' rounding allows, and the command runs."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from test_attention_layer_gpu import ROOT, _lengths, example   # noqa: F401,E402


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("norms", [False, True])
@pytest.mark.parametrize("batch,prompt,chunk", [(1, 40, 40), (3, 50, 17), (2, 300, 128)])
def test_against_the_16_bit_prompt(example, batch, prompt, chunk, norms, kind):   # noqa: F811
    layer = example.AttentionLayer(hidden=512, heads=8, kv_heads=2, dim=64, context=512, norms=norms)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(batch, prompt + 1, 512, generator=g, device="cuda").bfloat16()
    whole = example.PagedCache(batch, prompt + 1, 2, 64)
    whole.lengths += prompt + 1
    want = layer.prefill(x.reshape(-1, 512), whole, _lengths(batch, prompt + 1)).view(batch, prompt + 1, 512)
    cls, dtype = {"bf16": (example.PagedCache, torch.bfloat16), "int8": (example.PagedCache8, torch.int8),
                  "e4m3": (example.PagedCache8, torch.float8_e4m3fn)}[kind]
    cache = cls(batch, prompt + 1, 2, 64, dtype=dtype, seed=9)
    # In norm over many elements a code's rounding is about 1 / sqrt(12) of its step.  int8: steps of 1 / 127 of the largest
    # of 16 x 64 about normal values, 4 sigma and rarely more: 0.9 % of the values.  e4m3: steps of 1/16 to 1/8 of the value:
    # 2.6 % on the mean.  Values carry it as it is, keys as an error of the scores of that times the score's size, about 1:
    # as much again, taken four times in all.
    code = {"bf16": 0.0, "int8": 0.009, "e4m3": 0.026}[kind] * 4
    for at in range(0, prompt, chunk):
        part = x[:, at:min(at + chunk, prompt)]
        cache.lengths += part.shape[1]
        got = layer.prefill(part.reshape(-1, 512), cache, _lengths(batch, part.shape[1])).view(batch, -1, 512)
        ref = want[:, at:at + part.shape[1]]
        assert (got - ref).norm() <= (1e-2 + code) * ref.norm()
    cache.lengths += 1
    y = layer.decode(x[:, -1].float().contiguous(), cache, _lengths(batch, 1))
    torch.cuda.synchronize()
    import q4_dequant_gemv_gb300 as q4k
    assert q4k.device_error_flags() == 0
    ref = want[:, -1]
    assert (y - ref).norm() <= (4 * 2.0 ** -8 + code) * ref.norm()


@pytest.mark.parametrize("flags", [["--cache", "int8"], ["--cache", "e4m3", "--norms"], ["--norms"]])
def test_command_runs(example, flags):   # noqa: F811
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "attention_layer.py"), "--batch", "2", "--prompt",
                        "300", "--steps", "4", *flags], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "error flags 0" in r.stdout
