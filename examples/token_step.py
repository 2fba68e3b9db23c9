"""A small decoder from token to token on the library's calls alone: embedding rows, layers (norm, NVFP4 linears, attention over a
paged cache, SiLU * mul), the head and the draw of the next token, the whole step in one CUDA graph.

Prompts are read in one chunk with NVFP4 activations (the norm hands its output to the W4A4 linears as codes); decode steps use the
W4A16 linears. The residual stream is kept in 32 bits.

    python examples/token_step.py [--steps 16] [--temperature 0.8 --top-k 40 --top-p 0.95 --min-p 0.01]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_04_gb300 as nv  # noqa: E402


class Decoder:
    """Hidden 512, 8 query heads of 64 on 2, two layers, random weights."""

    hidden, inner, heads, kv_heads, dim, layers, vocab, page, pages, max_pages = 512, 1024, 8, 2, 64, 2, 3000, 16, 64, 16

    def __init__(self, batch: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def linear(n, k):
            q = nv.quantize(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5)
            return q, nv.prepack_scales(q)

        def gain(n):
            return (1 + 0.1 * torch.randn(n, generator=g, device="cuda")).bfloat16()

        width = (self.heads + 2 * self.kv_heads) * self.dim
        self.embedding = torch.randn(self.vocab, self.hidden, generator=g, device="cuda")
        self.blocks = [dict(norm1=gain(self.hidden), norm2=gain(self.hidden), norm_q=gain(self.dim), norm_k=gain(self.dim), qkv=linear(width, self.hidden),
                            out=linear(self.hidden, self.heads * self.dim), up=linear(2 * self.inner, self.hidden), down=linear(self.hidden, self.inner),
                            cache=nv.kv_cache(self.pages, self.kv_heads, self.page, self.dim),
                            table=torch.full((batch, self.max_pages), -1, dtype=torch.int32, device="cuda"),
                            refs=torch.zeros(self.pages, dtype=torch.int32, device="cuda")) for _ in range(self.layers)]
        self.norm = gain(self.hidden)
        self.head = linear(self.vocab, self.hidden)[0]

    def __call__(self, tokens, lens, start=None, max_new=1, workspace=None):
        """tokens int [T] at the ends of sequences of lengths lens -> logits bf16 [T][vocab]."""
        stream = self.embedding[tokens]                          # fp32, the stream that layers add to
        prompt = start is not None
        y = torch.zeros(len(tokens), self.hidden, dtype=torch.bfloat16, device="cuda")
        for b in self.blocks:
            nv.kv_reserve(b["table"], lens, b["refs"], self.page, start=start, max_new=max_new)
            qkv = self.linear(y, stream, b["norm1"], b["qkv"], prompt).view(len(tokens), -1, self.dim)
            q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
            nv.rms_norm(q, b["norm_q"], out=q)                   # each head by itself, in place
            nv.rms_norm(k, b["norm_k"], out=k)
            nv.kv_append(b["cache"], k, v, b["table"], lens, start=start, max_new=max_new)
            o = nv.paged_attention(q, b["cache"], b["table"], lens, start=start, max_new=max_new, workspace=workspace)
            y = nv.gemm_w4a16(o.view(len(tokens), -1), b["out"][0])
            if prompt:
                up = self.linear(y, stream, b["norm2"], b["up"], True).float()
                h = (torch.nn.functional.silu(up[:, :self.inner]) * up[:, self.inner:]).bfloat16()
            else:
                h, _ = nv.rms_norm(y, b["norm2"], residual=stream, residual_out=stream)
                h = nv.gemm_w4a16_silu_mul(h, b["up"][0])
            y = nv.gemm_w4a16(h, b["down"][0])
        y, _ = nv.rms_norm(y, self.norm, residual=stream, residual_out=stream)
        return nv.gemm_w4a16(y, self.head)

    @staticmethod
    def linear(y, stream, gain, weight, prompt):
        """stream += y, and the linear of its norm."""
        if prompt:
            q, _ = nv.rms_norm_quantize(y, gain, residual=stream, residual_out=stream)
            return nv.gemm_w4a4(q, weight[1])
        h, _ = nv.rms_norm(y, gain, residual=stream, residual_out=stream)
        return nv.gemm_w4a16(h, weight[0])


def run(steps: int = 16, temperature: float = 0.8, top_k: int = 40, top_p: float = 0.95, min_p: float = 0.01, graph: bool = True):
    """Tokens [1 + steps][sequences] that follow three prompts, and their probabilities."""
    prompts = [[5, 17, 200, 31], list(range(100, 137)), [2999]]
    n = len(prompts)
    model = Decoder(n)
    settings = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    uniform = torch.rand(1 + steps, n, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
    u = uniform[0].clone()

    lens = ints([len(p) for p in prompts])
    start = ints([0, *torch.tensor([len(p) for p in prompts]).cumsum(0).tolist()])
    logits = model(ints([t for p in prompts for t in p]), lens, start=start, max_new=max(map(len, prompts)))
    token, prob = nv.sample(logits[start[1:].long() - 1], u, **settings)
    out, probs = [token.clone()], [prob.clone()]

    workspace = nv.attention_workspace(n, 1, model.heads, model.kv_heads, model.dim)
    state = [lens, *(t for b in model.blocks for t in (b["table"], b["refs"]))]

    def step():
        lens.add_(1)
        return nv.sample(model(token, lens, workspace=workspace), u, **settings)

    if graph:
        saved = [t.clone() for t in state]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                               # warm up (allocations), then take it back
            for t, s in zip(state, saved):
                t.copy_(s)
            side.synchronize()
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured, stream=side):
                result = step()
        torch.cuda.current_stream().wait_stream(side)
    for i in range(steps):
        u.copy_(uniform[1 + i])
        if graph:
            captured.replay()
        else:
            result = step()
        token.copy_(result[0])
        out.append(result[0].clone())
        probs.append(result[1].clone())
    assert nv.read_device_status() == nv.OK
    return torch.stack(out), torch.stack(probs)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--top-k", type=int, default=40)
    ap.add_argument("--top-p", type=float, default=0.95)
    ap.add_argument("--min-p", type=float, default=0.01)
    a = ap.parse_args()
    tokens, probs = run(a.steps, a.temperature, a.top_k, a.top_p, a.min_p)
    for s in range(tokens.shape[1]):
        print(f"sequence {s}:", " ".join(f"{int(t)} ({float(p):.2f})" for t, p in zip(tokens[:, s], probs[:, s])))
