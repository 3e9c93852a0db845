"""One attention layer of a Q4_K model on the GPU: the quantized products with the rotation, the paged cache and the
attention between them, as an engine runs them.

    python examples/attention_layer.py [--batch 4] [--prompt 1000] [--steps 16] [--cache bf16|int8|e4m3] [--norms]

A prompt goes through in chunks (bf16 activations, tensor-core products), then tokens are decoded one by one from a
CUDA graph in which every launch is a programmatic dependent of the one before.  The shapes are those of a
Qwen2.5-7B layer (28 query heads, 4 cache heads of 128, hidden size 3584); weights and activations are synthetic."""
import argparse
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import q4_dequant_gemv_gb300 as q4k  # noqa: E402
import synth  # noqa: E402


class PagedCache:
    """Keys and values of up to `batch` sequences in pages handed out in a shuffled order; what the calls read of it
    (page table, lengths) lives on the device."""

    def __init__(self, batch, capacity, heads, dim, page=16, dtype=torch.bfloat16, seed=0):
        per = -(-capacity // page)
        self.k, self.v = (torch.zeros(batch * per, page, heads, dim, dtype=dtype, device="cuda") for _ in range(2))
        order = torch.randperm(batch * per, generator=torch.Generator().manual_seed(seed))
        self.pages = order.to(torch.int32).view(batch, per).cuda()
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def args(self, start):
        return self.k, self.v, self.pages, start, self.lengths

    def append(self, k, v, q, start, table, norms, q_out=None, q_dtype=None, pdl=False):
        """New keys and values of as many tokens of each sequence into the cache, the keys and queries normed by `norms`
        (two weights, or None) and turned -> the queries."""
        if norms is None:
            return q4k.kv_append(k, v, *self.args(start), table=table, q=q, q_out=q_out, q_dtype=q_dtype, pdl=pdl)
        n = q.shape[0] // self.lengths.shape[0]
        pos = (self.lengths[:, None] - n + torch.arange(n, dtype=torch.int32, device="cuda")).flatten()
        q, k = q4k.norm_rope(q, k, pos, table, *norms, q_out, out_dtype=q_dtype, pdl=pdl)
        q4k.kv_append(k, v.to(k.dtype), *self.args(start), pdl=pdl)     # (nothing left to turn)
        return q

    def attend(self, q, start, **kw):
        return q4k.paged_attention(q, *self.args(start), **kw)


class PagedCache8(PagedCache):
    """The same in 8 bits: codes, and a scale for each block of tokens and head."""

    def __init__(self, batch, capacity, heads, dim, page=16, dtype=torch.int8, block=None, seed=0):
        super().__init__(batch, capacity, heads, dim, page, dtype, seed)
        self.k_scale, self.v_scale = (torch.zeros(self.k.shape[0], page // (block or page), heads, device="cuda") for _ in range(2))

    def args(self, start):
        return self.k, self.v, self.k_scale, self.v_scale, self.pages, start, self.lengths

    def append(self, k, v, q, start, table, norms, q_out=None, q_dtype=None, pdl=False):
        q_weight, k_weight = norms or (None, None)          # (in the same launch here)
        return q4k.kv_append8(k, v, *self.args(start), table=table, q=q, q_out=q_out, q_dtype=q_dtype, q_weight=q_weight,
                              k_weight=k_weight, pdl=pdl)

    def attend(self, q, start, **kw):
        return q4k.paged_attention8(q, *self.args(start), **kw)


class AttentionLayer:
    def __init__(self, hidden=3584, heads=28, kv_heads=4, dim=128, context=32768, base=1000000.0, seed=1, norms=False):
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim
        # synthetic weights with a mean near 0
        def weights(rows, cols, tag):
            w = synth.q4k_weights(rows, cols, (seed, tag)).copy()
            w.reshape(rows, cols // 256, 144)[:, :, 0:4] = 0
            h = w.reshape(rows, cols // 256, 144)[:, :, 0:4].copy().view("float16")
            h[..., 0], h[..., 1] = 0.06 / (24 * cols ** 0.5), 0.45 / (24 * cols ** 0.5)
            w.reshape(rows, cols // 256, 144)[:, :, 0:4] = h.view("uint8")
            return torch.from_numpy(w).cuda()

        self.wq, self.wk, self.wv = weights(heads * dim, hidden, 1), weights(kv_heads * dim, hidden, 2), weights(kv_heads * dim, hidden, 3)
        self.wo = weights(hidden, heads * dim, 4)
        self.table = q4k.rope_table(context, dim, base)
        self.norms = None       # weights of the query and key heads' norms, where the model has them
        if norms:
            g = torch.Generator().manual_seed(seed)
            self.norms = tuple((1 + 0.1 * torch.randn(dim, generator=g)).cuda() for _ in range(2))

    def _heads(self, y, n):
        return y.view(-1, n, self.dim)

    def prefill(self, x, cache, start):
        """x bf16 [tokens, hidden]: the sequences' next chunks, cache.lengths already counting them -> fp32."""
        q, k, v = (q4k.gemm_prefill(w, x) for w in (self.wq, self.wk, self.wv))
        q = cache.append(self._heads(k, self.kv_heads), self._heads(v, self.kv_heads), self._heads(q, self.heads), start, self.table,
                         self.norms, q_dtype=torch.bfloat16)
        y = cache.attend(q, start)
        return q4k.gemm_prefill(self.wo, y.view(x.shape[0], -1))

    def decode(self, x, cache, start, pdl=True):
        """x fp32 [sequences, hidden]: a token each -> fp32."""
        q, k, v = q4k.gemv_grouped([self.wq, self.wk, self.wv], x, pdl=pdl)
        q = self._heads(q, self.heads)
        q = cache.append(self._heads(k, self.kv_heads), self._heads(v, self.kv_heads), q, start, self.table, self.norms, q_out=q, pdl=pdl)
        y = cache.attend(q, start, pdl=pdl)
        return q4k.gemv(self.wo, y.view(x.shape[0], -1), pdl=pdl)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--chunk", type=int, default=512)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--cache", choices=("bf16", "int8", "e4m3"), default="bf16")
    ap.add_argument("--norms", action="store_true", help="norms of the query and key heads")
    a = ap.parse_args()
    layer = AttentionLayer(norms=a.norms)
    kind, dtype = {"bf16": (PagedCache, torch.bfloat16), "int8": (PagedCache8, torch.int8), "e4m3": (PagedCache8, torch.float8_e4m3fn)}[a.cache]
    cache = kind(a.batch, a.prompt + a.steps + 1, layer.kv_heads, layer.dim, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(a.batch, a.prompt, layer.hidden, generator=g, device="cuda").bfloat16()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for at in range(0, a.prompt, a.chunk):
        part = x[:, at:at + a.chunk].reshape(-1, layer.hidden)
        n = part.shape[0] // a.batch
        cache.lengths += n
        y = layer.prefill(part, cache, torch.arange(a.batch + 1, dtype=torch.int32, device="cuda") * n)
    torch.cuda.synchronize()
    print(f"prompt: {a.batch} x {a.prompt} tokens in {1e3 * (time.perf_counter() - t):.2f} ms, |y| {y.abs().mean():.3f}")

    start = torch.arange(a.batch + 1, dtype=torch.int32, device="cuda")
    tok = torch.randn(a.batch, layer.hidden, generator=g, device="cuda")
    cache.lengths += 1
    layer.decode(tok, cache, start)       # first launches outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.decode(tok, cache, start)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()                    # the graph reads the lengths from the device
        cache.lengths += 1
    torch.cuda.synchronize()
    print(f"decode: {a.steps} steps of {a.batch} tokens, {1e6 * (time.perf_counter() - t) / a.steps:.1f} us a step, "
          f"|y| {out.abs().mean():.3f}, error flags {q4k.device_error_flags()}")


if __name__ == "__main__":
    main()
