"""The example's attention layer: decoding a token after a prompt gives what the prompt with that token gives, whatever
the chunks, and the command runs."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import attention_layer
    finally:
        sys.path.pop(0)
    torch.cuda.set_device(0)
    return attention_layer


def _lengths(batch, n):
    return torch.arange(batch + 1, dtype=torch.int32, device="cuda") * n


@pytest.mark.parametrize("batch,prompt,chunk", [(1, 40, 40), (3, 50, 17), (2, 300, 128)])
def test_decode_continues_the_prompt(example, batch, prompt, chunk):
    layer = example.AttentionLayer(hidden=512, heads=8, kv_heads=2, dim=64, context=512)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(batch, prompt + 1, 512, generator=g, device="cuda").bfloat16()
    whole = example.PagedCache(batch, prompt + 1, 2, 64)
    whole.lengths += prompt + 1
    want = layer.prefill(x.reshape(-1, 512), whole, _lengths(batch, prompt + 1)).view(batch, prompt + 1, 512)
    cache = example.PagedCache(batch, prompt + 1, 2, 64, seed=9)
    for at in range(0, prompt, chunk):
        part = x[:, at:min(at + chunk, prompt)]
        cache.lengths += part.shape[1]
        got = layer.prefill(part.reshape(-1, 512), cache, _lengths(batch, part.shape[1])).view(batch, -1, 512)
        # the same roundings, in tiles that begin elsewhere: fp32 sums in another order
        ref = want[:, at:at + part.shape[1]]
        assert (got - ref).norm() <= 1e-2 * ref.norm()
    cache.lengths += 1
    y = layer.decode(x[:, -1].float().contiguous(), cache, _lengths(batch, 1))
    torch.cuda.synchronize()
    import q4_dequant_gemv_gb300 as q4k
    assert q4k.device_error_flags() == 0
    # the prompt's path rounds the weights once to fp16, and q, the softmax weights and the attention's output
    # to bf16 (2^-8 each at most); the decode path does not
    ref = want[:, -1]
    assert (y - ref).norm() <= 4 * 2.0 ** -8 * ref.norm()


def test_command_runs(example):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "attention_layer.py"), "--batch", "2", "--prompt",
                        "300", "--steps", "4"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "error flags 0" in r.stdout
