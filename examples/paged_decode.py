"""A decoder layer's attention block as a serving loop runs it: NVFP4 qkv and output projections (W4A16) around a paged key-value cache.

Three ragged prompts are read in one chunk each, the second is sampled two ways (forked), every sequence decodes a few tokens in a CUDA
graph (reserve, append, attention under a sliding window with sinks), the parent is released, and the pool is compacted in the middle
of decoding.

    python examples/paged_decode.py [--kv e4m3] [--steps 24]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_04_gb300 as nv  # noqa: E402


class Layer:
    """One attention block: hidden 1024, 8 query heads of 128 on 2 kv heads."""

    hidden, heads, kv_heads, dim, page, pages, max_pages = 1024, 8, 2, 128, 16, 256, 64

    def __init__(self, kv: str, window: int, sinks: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = (self.heads + 2 * self.kv_heads) * self.dim
        self.w_qkv = nv.quantize(torch.randn(rows, self.hidden, generator=g, device="cuda") * 0.04)
        self.w_out = nv.quantize(torch.randn(self.hidden, self.heads * self.dim, generator=g, device="cuda") * 0.04)
        scale = torch.full((self.kv_heads,), 1 / 64, device="cuda")
        self.cache = nv.kv_cache(self.pages, self.kv_heads, self.page, self.dim,
                                 torch.float8_e4m3fn if kv == "e4m3" else torch.bfloat16, scale, scale)
        self.window, self.sinks = window, sinks

    def __call__(self, x, table, lens, start=None, max_new=1, workspace=None):
        """x bf16 [tokens][hidden] -> the same after attention and the output projection; keys and values go into the cache."""
        qkv = nv.gemm_w4a16(x, self.w_qkv).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        nv.kv_append(self.cache, k, v, table, lens, start=start, max_new=max_new)
        o = nv.paged_attention(q, self.cache, table, lens, start=start, max_new=max_new, window=self.window, sinks=self.sinks,
                               workspace=workspace)
        return nv.gemm_w4a16(o.view(x.shape[0], -1), self.w_out)


def run(kv: str = "bf16", steps: int = 24, window: int = 128, sinks: int = 4):
    """Returns (outputs [steps][sequences][hidden], the same from prompts read again in one piece): they agree."""
    torch.manual_seed(1)
    prompts = [37, 150, 5]
    n_seq = len(prompts) + 2                       # room for two forks of the second
    layer = Layer(kv, window, sinks)
    table = torch.full((n_seq, layer.max_pages), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
    refs = torch.zeros(layer.pages, dtype=torch.int32, device="cuda")
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")

    # prompts: pages for them, keys and values into the cache, attention
    x = torch.randn(sum(prompts), layer.hidden, device="cuda").bfloat16()
    rows = len(prompts)
    start = ints([0, *torch.tensor(prompts).cumsum(0).tolist()])
    lens[:rows] = ints(prompts)
    nv.kv_reserve(table[:rows], lens[:rows], refs, layer.page, start=start, max_new=max(prompts))
    layer(x, table[:rows], lens[:rows], start=start, max_new=max(prompts))

    # sample the second prompt two ways, and let the prompt itself go
    nv.kv_fork(layer.cache, table, lens, refs, ints([1, 1]), ints([3, 4]))
    nv.kv_release(table, lens, refs, ints([1]))
    alive = [0, 2, 3, 4]
    prompt_of = [0, 2, 1, 1]
    table_a, lens_a = table[alive], lens[alive]    # the batch of the decode loop

    # one step, captured: every length lives on the device
    tokens = torch.randn(steps, len(alive), layer.hidden, device="cuda").bfloat16()
    token = tokens[0].clone()
    ws = nv.attention_workspace(len(alive), 1, layer.heads, layer.kv_heads, layer.dim)

    def step():
        lens_a.add_(1)
        nv.kv_reserve(table_a, lens_a, refs, layer.page)
        return layer(token, table_a, lens_a, workspace=ws)

    saved = [t.clone() for t in (table_a, lens_a, refs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                     # warm up (allocations), then take it back
        for t, s in zip((table_a, lens_a, refs), saved):
            t.copy_(s)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = step()
    torch.cuda.current_stream().wait_stream(side)
    out = []
    for i in range(steps):
        token.copy_(tokens[i])
        graph.replay()
        out.append(y.clone())
        if i == steps // 2:                        # the pool is tidied up between two steps
            live = nv.kv_compact(layer.cache, table_a, refs)
            assert int(live) == int((refs > 0).sum()) and not refs[int(live):].any()
    assert nv.read_device_status() == nv.OK

    # the same sequences read again from the start, prompt and tokens in one chunk
    again = Layer(kv, window, sinks)
    n_new = [prompts[p] + steps for p in prompt_of]
    offsets = torch.tensor([0, *prompts]).cumsum(0).tolist()
    pieces = [torch.cat([x[offsets[p]:offsets[p + 1]], tokens[:, b]]) for b, p in enumerate(prompt_of)]
    start = ints([0, *torch.tensor(n_new).cumsum(0).tolist()])
    table2 = torch.full((len(alive), layer.max_pages), -1, dtype=torch.int32, device="cuda")
    refs2 = torch.zeros(layer.pages, dtype=torch.int32, device="cuda")
    nv.kv_reserve(table2, ints(n_new), refs2, layer.page, start=start, max_new=max(n_new))
    whole = again(torch.cat(pieces), table2, ints(n_new), start=start, max_new=max(n_new))
    last = torch.stack([whole[int(e) - steps:int(e)] for e in start[1:]], dim=1)
    return torch.stack(out), last


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--kv", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--steps", type=int, default=24)
    a = ap.parse_args()
    stepwise, at_once = run(a.kv, a.steps)
    err = ((stepwise.float() - at_once.float()).norm() / at_once.float().norm()).item()
    print(f"{a.steps} decode steps of {stepwise.shape[1]} sequences, {a.kv} cache: relative difference to one chunk {err:.2e}")
