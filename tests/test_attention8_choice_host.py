"""The form that the library takes by itself for a call over an 8-bit cache, over a runtime that runs nothing: widening the
cache counts for the many-rows form."""
import pytest

pytest.importorskip("torch")
from fake_runtime import fake, fake_path   # noqa: F401,E402
from test_attention_abi import _attention   # noqa: E402
from test_cache8_abi import _bind, _cache8   # noqa: E402


def _widens(fake, batch, tokens, positions, heads, kv_heads, flags=0):   # noqa: F811
    """Whether a bf16 call of `tokens` new tokens a sequence widens its cache (heads of 128, pages of 64, blocks of 16)."""
    L, D, pages = _bind(fake), 128, -(-positions // 64)
    c = _cache8(size=64, heads=kv_heads, dim=D, block=16, kh=D, ks=D * kv_heads, kp=64 * D * kv_heads, vh=D, vs=D * kv_heads,
                vp=64 * D * kv_heads, pages=1 << 16, row=pages, most=pages, batch=batch, tokens=batch * tokens)
    a = _attention(heads=heads, qt=D * heads, qh=D, ot=D * heads, oh=D, flags=flags)
    assert L.q4k_paged_attention8(c, a, 0) == 0
    got = fake.launches()
    assert got
    return any(b"widen" in x.kernel for x in got)


@pytest.mark.parametrize("batch,tokens,positions,heads,kv_heads,many", [
    # measured, us: the fastest few-rows form and the many-rows form
    (64, 4, 512, 28, 4, False),       # 38, 82
    (4, 8, 8064, 32, 8, False),       # 50, 80
    (16, 8, 2048, 32, 8, False),      # 49, 86
    (64, 8, 2048, 32, 8, False),      # 195, 287
    (16, 4, 32064, 28, 4, False),     # 288, 463
    (4, 32, 8064, 28, 4, True),       # 146, 59
    (16, 32, 2048, 32, 8, True),      # 200, 100
    (1, 2048, 16384, 32, 8, True),    # 4030, 397
    (1, 1, 131072, 32, 8, False),
])
def test_widening_counts(fake, batch, tokens, positions, heads, kv_heads, many):   # noqa: F811
    assert _widens(fake, batch, tokens, positions, heads, kv_heads) is many
    assert _widens(fake, batch, tokens, positions, heads, kv_heads, 7 << 8)
