"""One attention block of a decoder, served with drafted trees:  python examples/tree_decode.py

The block's projections are unstructured-sparse matrices (us_spmm_f16), its keys
and values a quantised paged cache.  Three requests prefill their prompts in
chunks, then each step
  1. projects a tree of drafted tokens per request     us_spmm_f16
  2. appends the drafts' keys and values               us_kv_write
  3. attends, each draft to the context and its own    us_attn_kv
     ancestors, and projects back                      us_spmm_f16
  4. keeps one root-to-leaf path                       us_kv_commit
The last tokens are decoded one at a time from a CUDA graph whose positions live
on the device.  Weights, prompts, drafts and the accepted paths are random (a model
would give them): what is shown is the calls.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bitmap_encoded_unstructured_ie_gb300 import binding as us  # noqa: E402


class Block:
    """out(attention(qkv(x))) with Hq query heads on Hkv key heads of D dimensions."""

    def __init__(self, hidden=512, Hq=8, Hkv=2, D=64, elem=us.US_I8, page=16, B=3, max_pages=20, sparsity=0.5, seed=0):
        self.hidden, self.Hq, self.Hkv, self.D, self.scale = hidden, Hq, Hkv, D, D ** -0.5
        g = self.gen = torch.Generator(device="cuda").manual_seed(seed)

        def sparse(rows, cols):
            w = torch.randn(rows, cols, generator=g, device="cuda") / (cols * (1 - sparsity)) ** 0.5
            w = w * (torch.rand(rows, cols, generator=g, device="cuda") >= sparsity)
            return us.us_encode(w.half(), 64, 64, us.US_F16, us.US_ORDER_ROW)

        self.qkv, self.out = sparse((Hq + 2 * Hkv) * D, hidden), sparse(hidden, Hq * D)
        # the requests' pages lie scattered in one pool
        table = torch.randperm(B * max_pages, generator=g, device="cuda").to(torch.int32).view(B, max_pages)
        self.cache = us.kv_cache(elem, D, Hkv, page, B * max_pages, table)
        self.ws = {}

    def product(self, E, x):
        n = x.shape[0]
        if (E.M, n) not in self.ws:
            self.ws[E.M, n] = us.workspace(us.US_OP_SPMM_F16, E, n)
        y = torch.empty(n, E.M, dtype=torch.float16, device="cuda")
        us.us_spmm_f16(E, x, n, y, self.ws[E.M, n])
        return y

    def forward(self, x, off, pos, mask, max_n):
        """Rows x of the requests' tokens (off, pos as in us_kv_write): appends, attends, projects."""
        T, kv = x.shape[0], self.Hq + self.Hkv
        qkv = self.product(self.qkv, x).view(T, kv + self.Hkv, self.D)
        us.us_kv_write(self.cache, qkv[:, self.Hq:kv], qkv[:, kv:], off, pos, max_n)
        o = torch.empty(T, self.Hq, self.D, dtype=torch.float16, device="cuda")
        if max_n not in self.ws:
            self.ws[max_n] = us.workspace_attn_kv(self.cache, self.Hq, max_n)
        us.us_attn_kv(self.cache, qkv[:, :self.Hq], off, pos, mask, max_n, self.scale, o, self.ws[max_n])
        return self.product(self.out, o.view(T, -1)), qkv, o


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(n):
    return ints([sum(n[:i]) for i in range(len(n) + 1)])


def tree_masks(parents):
    """Each draft sees itself and its ancestors: bit j of its word for draft j."""
    masks = []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
    return masks


def signed(words):
    """64-bit words as int64 values."""
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")


def run(steps=3, single=4, prompts=(37, 150, 16), chunk=64, drafts=(16, 9, 21), watch=None, **block):
    """Prefill, `steps` trees, `single` tokens one at a time; returns the block, the requests' lengths and
    the last outputs.  watch(block, **call), if given, is called after each attention and each commit."""
    blk = Block(B=len(prompts), **block)
    B, rng = len(prompts), torch.Generator().manual_seed(1)
    length, x_of = [0] * B, lambda n: torch.randn(n, blk.hidden, generator=blk.gen, device="cuda").half()

    watch = watch or (lambda block, **call: None)

    def forward(n, parents=None):
        mask = signed([m for p in parents for m in tree_masks(p)]) if parents else None
        y, qkv, o = blk.forward(x_of(sum(n)), offsets(n), ints(length), mask, max(n))
        watch(blk, qkv=qkv, o=o, n=n, pos=list(length), parents=parents)
        return y

    while any(length[b] < prompts[b] for b in range(B)):                      # the prompts, chunk by chunk
        n = [min(chunk, prompts[b] - length[b]) for b in range(B)]
        y = forward(n)
        length = [length[b] + n[b] for b in range(B)]

    for _ in range(steps):                                                    # trees
        parents = [[-1] + [int(torch.randint(i, (1,), generator=rng)) for i in range(1, n)] for n in drafts]
        y = forward(list(drafts), parents)
        paths = []
        for p in parents:
            leaf = int(torch.randint(len(p), (1,), generator=rng))
            path = [leaf]
            while p[path[-1]] >= 0:
                path.append(p[path[-1]])
            paths.append(path[::-1])
        acc = ints([j for path in paths for j in path])
        us.us_kv_commit(blk.cache, offsets([len(p) for p in paths]), acc, ints(length), max(map(len, paths)))
        watch(blk, paths=paths, pos=list(length))
        length = [length[b] + len(paths[b]) for b in range(B)]

    # single tokens: one graph, replayed with the positions it moves on itself
    x, off, pos = x_of(B), offsets([1] * B), ints(length)
    blk.forward(x, off, pos, None, 1)                                         # makes the workspaces
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, qkv, o = blk.forward(x, off, pos, None, 1)
        pos += 1
    for _ in range(single):
        x.copy_(x_of(B))
        graph.replay()
        watch(blk, qkv=qkv, o=o, n=[1] * B, pos=list(length), parents=None)
        length = [n + 1 for n in length]
    status = us.us_get_last_device_status()
    assert status == us.US_OK, f"device status {status}"
    return blk, length, y


def main():
    blk, length, y = run()
    K, V = (torch.empty(sum(length), blk.Hkv, blk.D, dtype=torch.float16, device="cuda") for _ in range(2))
    us.us_kv_read(blk.cache, offsets(length), ints([0] * len(length)), max(length), K, V)     # the whole cache as fp16
    print("requests hold", length, "positions; last outputs", tuple(y.shape), "rms %.3f;" % y.float().pow(2).mean().sqrt(),
          "cache rms: keys %.3f, values %.3f" % (K.float().pow(2).mean().sqrt(), V.float().pow(2).mean().sqrt()))


if __name__ == "__main__":
    main()
