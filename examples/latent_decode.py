"""One latent attention block of a decoder, served:  python examples/latent_decode.py

Every token leaves one latent row and one rotated key, which all heads share, in a paged
cache.  Its projections are unstructured-sparse matrices (us_spmm_f16); a token's queries and
outputs pass through the head's part of one of them, dense, by einsum.  Three requests
prefill their prompts in chunks, then decode single tokens:
  1. pages for the new tokens                           us_kv_reserve
  2. queries, latent rows; their rotation, the cache    us_spmm_f16, us_norm_rope, us_lat_write
  3. prompts: the context's latent rows are read and expanded to each head's keys and
     values, and the chunk attends to them              us_lat_read, us_spmm_f16, us_attn_rows
     tokens: the queries are taken into the latent space instead, attend there, and the
     outputs are taken back                             us_attn_lat
Single tokens run from a CUDA graph in which pages, positions and lengths move on the
device.  Weights and inputs are random: what is shown is the calls.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bitmap_encoded_unstructured_ie_gb300 import binding as us  # noqa: E402


class Block:
    """H heads of Dn + 64 dimensions (values of Dn) over latent rows of Dc + 64."""

    def __init__(self, hidden=512, H=4, Dn=64, Dc=256, page=16, B=3, max_pages=20, num_pages=40, sparsity=0.5, seed=0):
        self.hidden, self.H, self.Dn, self.Dc, self.scale = hidden, H, Dn, Dc, (Dn + 64) ** -0.5
        g = self.gen = torch.Generator(device="cuda").manual_seed(seed)

        def sparse(rows, cols):
            w = torch.randn(rows, cols, generator=g, device="cuda") / (cols * (1 - sparsity)) ** 0.5
            w = (w * (torch.rand(rows, cols, generator=g, device="cuda") >= sparsity)).half()
            return w, us.us_encode(w, 64, 64, us.US_F16, us.US_ORDER_ROW)

        self.wq, self.q = sparse(H * (Dn + 64), hidden)
        self.wc, self.c = sparse(Dc + 64, hidden)
        self.wkv, self.kv = sparse(H * 2 * Dn, Dc)                            # each head's key, then its value
        self.wo, self.out = sparse(hidden, H * Dn)
        self.norm = (1 + 0.2 * torch.randn(Dc, generator=g, device="cuda")).half()
        freq = 10000.0 ** (-2.0 * torch.arange(32, dtype=torch.float64) / 64)
        self.rope = us.Rope(us.US_ROPE_PAIRS, us.rope_freq(freq).cuda())
        self.pool = us.kv_pool(page, num_pages, B, max_pages)
        self.cache = us.lat_cache(Dc, 64, page, num_pages, self.pool.page_table)
        self.ws = {}

    def product(self, E, x):
        n, y = x.shape[0], None
        for lo in range(0, n, 2048):                                          # (us_spmm_f16 takes up to 2048 tokens)
            part = x[lo:lo + 2048]
            if (E.M, E.K, len(part)) not in self.ws:
                self.ws[E.M, E.K, len(part)] = us.workspace(us.US_OP_SPMM_F16, E, len(part))
            y = torch.empty(n, E.M, dtype=torch.float16, device="cuda") if y is None else y
            us.us_spmm_f16(E, part, len(part), y[lo:lo + 2048], self.ws[E.M, E.K, len(part)])
        return y

    def enter(self, x, off, pos, max_n):
        """Queries of rows x (turned), whose latent rows enter the cache."""
        T = x.shape[0]
        q = self.product(self.q, x).view(T, self.H, self.Dn + 64)
        part = q[..., self.Dn:]
        us.us_norm_rope(self.rope, part, None, part, None, None, None, off, pos, None, max_n)
        us.us_lat_write(self.cache, self.rope, self.product(self.c, x), self.norm, off, pos, None, max_n)
        return q

    def chunk(self, x, off, pos, max_n, kv_off, S, max_kv):
        """Rows x of prompts, attended to in the expanded form."""
        T, H, Dn = x.shape[0], self.H, self.Dn
        q = self.enter(x, off, pos, max_n)
        rows = torch.empty(S, self.Dc + 64, dtype=torch.float16, device="cuda")
        us.us_lat_read(self.cache, kv_off, torch.zeros_like(pos), max_kv, rows)
        kv = self.product(self.kv, rows[:, :self.Dc].contiguous()).view(S, H, 2 * Dn)
        o = torch.empty(T, H, Dn, dtype=torch.float16, device="cuda")
        ws = us.workspace_attn_rows(Dn, 64, Dn, H, len(off) - 1, max_n)
        us.us_attn_rows(q, kv[..., :Dn], rows[:, self.Dc:], kv[..., Dn:], off, kv_off, max_n, self.scale, o, ws)
        return self.product(self.out, o.view(T, -1)), q, o

    def token(self, x, off, pos):
        """One token of every request, attended to in the latent space."""
        T, H, Dn = x.shape[0], self.H, self.Dn
        q = self.enter(x, off, pos, 1)
        w = self.wkv.view(H, 2 * Dn, self.Dc)
        inner = torch.empty(T, H, self.Dc + 64, dtype=torch.float16, device="cuda")
        inner[..., :self.Dc] = torch.einsum("thd,hdc->thc", q[..., :Dn], w[:, :Dn])
        inner[..., self.Dc:] = q[..., Dn:]
        y = torch.empty(T, H, self.Dc, dtype=torch.float16, device="cuda")
        if "attn" not in self.ws:
            self.ws["attn"] = us.workspace_attn_lat(self.cache, H, 1)
        us.us_attn_lat(self.cache, inner, off, pos, None, 1, self.scale, y, self.ws["attn"])
        o = torch.einsum("thc,hdc->thd", y, w[:, Dn:]).contiguous()
        return self.product(self.out, o.view(T, -1)), q, o


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(n):
    return ints([sum(n[:i]) for i in range(len(n) + 1)])


def run(single=20, prompts=(37, 150, 16), chunk=64, watch=None, **block):
    """Prefill, then `single` tokens; returns the block, the requests' lengths and the last outputs.
    watch(block, x=, o=, n=, pos=), if given, is called after each attention."""
    blk = Block(B=len(prompts), **block)
    B, length = len(prompts), [0] * len(prompts)
    x_of = lambda n: torch.randn(n, blk.hidden, generator=blk.gen, device="cuda").half()  # noqa: E731
    watch = watch or (lambda block, **call: None)
    while any(length[b] < prompts[b] for b in range(B)):                      # the prompts, chunk by chunk
        n = [min(chunk, prompts[b] - length[b]) for b in range(B)]
        kv = [a + b for a, b in zip(length, n)]
        us.us_kv_reserve(blk.pool, ints(kv))
        x = x_of(sum(n))
        y, q, o = blk.chunk(x, offsets(n), ints(length), max(max(n), 1), offsets(kv), sum(kv), max(kv))
        watch(blk, x=x, o=o, n=n, pos=list(length))
        length = kv

    # single tokens: one graph, replayed with the positions it moves on itself
    x, off, pos, lens = x_of(B), offsets([1] * B), ints(length), ints(length) + 1
    us.us_kv_reserve(blk.pool, lens)
    blk.token(x, off, pos)                                                    # makes the workspaces
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        us.us_kv_reserve(blk.pool, lens)
        y, q, o = blk.token(x, off, pos)
        pos += 1
        lens += 1
    for _ in range(single):
        x.copy_(x_of(B))
        graph.replay()
        watch(blk, x=x, o=o, n=[1] * B, pos=list(length))
        length = [n + 1 for n in length]
    status = us.us_get_last_device_status()
    assert status == us.US_OK, f"device status {status}"
    return blk, length, y


def main():
    blk, length, y = run()
    print("requests hold", length, "positions on", blk.pool.held.tolist(), "pages,", int(blk.pool.free_count), "free; last outputs",
          tuple(y.shape), "rms %.3f" % y.float().pow(2).mean().sqrt())


if __name__ == "__main__":
    main()
