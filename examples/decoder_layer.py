"""One decoder layer served with this library's operators, prompt and decoding alike.

    python examples/decoder_layer.py                       # 4096 channels, 32 heads, 4 sequences
    python examples/decoder_layer.py --hidden 12288 --heads 96 --prompt 500

The layer is OPT's without biases (normalisation, attention, normalisation, a ReLU MLP; random
weights): the QKV product runs on pruned weights (lscd_spmm), new keys and values go into a paged 8-bit
cache (lscd_cache_write), attention reads it (lscd_attention), and the output projection and the MLP run
on 4-bit weights (lscd_quant_linear).  A batch of prompts of different lengths goes through in one call,
then every sequence decodes one token at a time, as one captured graph that is replayed.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import unstructured_sparse_skinny_amd as L  # noqa: E402


def quantise_weights(w, group=128):
    """4-bit codes, scales and zero points of w [M][K], nearest over each row and group (K a multiple of group)."""
    M, K = w.shape
    g = w.float().view(M, K // group, group)
    low, high = g.amin(2).clamp(max=0), g.amax(2).clamp(min=0)
    scale = ((high - low) / 15).clamp(min=1e-8).to(w.dtype)
    zero = torch.round(-low / scale.float()).clamp(0, 15)
    code = (torch.round(g / scale.float()[..., None]) + zero[..., None]).clamp(0, 15).view(M, K).to(torch.uint8)
    return code[:, 0::2] | code[:, 1::2] << 4, scale, zero.to(torch.uint8)


class Layer:
    def __init__(self, hidden=4096, heads=32, sparsity=0.7, pages=256, page=16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(m, k):
            return (torch.randn((m, k), generator=g, device=device) * k ** -0.5).half()

        self.hidden, self.heads, self.dim, self.page = hidden, heads, hidden // heads, page
        qkv = weight(3 * hidden, hidden)
        qkv *= torch.rand(qkv.shape, generator=g, device=device) >= sparsity
        self.qkv = L.lscd_encode_device(qkv)
        self.dense = {"qkv": qkv}
        for name, m, k in (("out", hidden, hidden), ("up", 4 * hidden, hidden), ("down", hidden, 4 * hidden)):
            codes, scale, zero = quantise_weights(weight(m, k))
            setattr(self, name, L.lscd_quant_encode(codes, scale, k, zero))
            self.dense[name] = torch.empty((m, k), device=device, dtype=torch.float16)
            L.lscd_quant_decode(getattr(self, name), self.dense[name])   # (what a plain layer is compared on)
        shape = (pages, heads, page, self.dim)
        self.cache = L.Cache(*(torch.zeros(shape, device=device, dtype=torch.float8_e4m3fn) for _ in range(2)),
                             *(torch.ones(shape[:3], device=device) for _ in range(2)))
        self.attention = L.lscd_attention_create(heads, heads, self.dim)

    def __call__(self, x, slots, start, length, table, b=None):
        """x [T][hidden]: new tokens of all sequences; slots: where each goes.  b: buffers to use again."""
        T, D = x.shape[0], self.hidden
        b = b if b is not None else self.buffers(T)
        L.lscd_spmm(self.qkv, torch.nn.functional.layer_norm(x, (D,)), b["qkv"])
        q, k, v = b["qkv"].view(T, 3, self.heads, self.dim).unbind(1)
        L.lscd_cache_write(self.cache, k, v, slots)
        L.lscd_attention(self.attention, self.cache, q, start, length, table, b["mixed"].view(T, self.heads, self.dim))
        L.lscd_quant_linear(self.out, b["mixed"], b["out"])
        x = x + b["out"]
        L.lscd_quant_linear(self.up, torch.nn.functional.layer_norm(x, (D,)), b["up"])
        L.lscd_quant_linear(self.down, torch.relu_(b["up"]), b["out"])
        return x + b["out"]

    def buffers(self, T):
        return {n: torch.empty((T, w * self.hidden), device="cuda", dtype=torch.float16)
                for n, w in (("qkv", 3), ("mixed", 1), ("out", 1), ("up", 4))}

    def plain(self, x, lengths):
        """The same layer on dense weights, whole sequences at once, in float32 (x [T][hidden], no cache)."""
        norm, w = torch.nn.functional.layer_norm, {n: t.float() for n, t in self.dense.items()}
        out, at, x = [], 0, x.float()
        for n in lengths:
            h = x[at:at + n]
            q, k, v = (norm(h, (self.hidden,)) @ w["qkv"].t()).view(n, 3, self.heads, self.dim).permute(1, 2, 0, 3)
            s = (q @ k.transpose(1, 2)) * self.dim ** -0.5
            s = s.masked_fill(torch.ones((n, n), device=s.device).triu(1).bool(), float("-inf"))
            h = h + (torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, -1) @ w["out"].t()
            out.append(h + torch.relu(norm(h, (self.hidden,)) @ w["up"].t()) @ w["down"].t())
            at += n
        return torch.cat(out)


def serve(layer, prompts, steps, seed=1):
    """Prompts (their lengths), then `steps` tokens for each sequence: all layer inputs and outputs, by sequence."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    S, page = len(prompts), layer.page
    wide = (max(prompts) + steps + page - 1) // page
    table = torch.arange(S * wide, device="cuda", dtype=torch.int32).view(S, wide)   # (an allocator's work)
    ints = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731

    def slots_of(positions):
        return ints([int(table[s, p // page]) * page + p % page for s, p in positions])

    x = torch.randn((sum(prompts), layer.hidden), generator=g, device="cuda").half()
    start = [0]
    for n in prompts:
        start.append(start[-1] + n)
    y = layer(x, slots_of([(s, p) for s, n in enumerate(prompts) for p in range(n)]), ints(start), ints(prompts), table)
    xs = [[x[start[s]:start[s + 1]]] for s in range(S)]
    ys = [[y[start[s]:start[s + 1]]] for s in range(S)]
    # decoding: one graph, its inputs updated between replays
    token, slots = torch.zeros((S, layer.hidden), device="cuda", dtype=torch.float16), slots_of(list(enumerate(prompts)))
    one, length, b = ints(list(range(S + 1))), ints([n + 1 for n in prompts]), layer.buffers(S)
    layer(token, slots, one, length, table, b)       # (once outside: libraries load their kernels)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(token, slots, one, length, table, b)
    for i in range(steps):
        token.copy_(torch.randn((S, layer.hidden), generator=g, device="cuda"))
        slots.copy_(slots_of([(s, n + i) for s, n in enumerate(prompts)]))
        length.copy_(ints([n + i + 1 for n in prompts]))
        graph.replay()
        for s in range(S):
            xs[s].append(token[s:s + 1].clone())
            ys[s].append(y[s:s + 1].clone())
    return [torch.cat(v) for v in xs], [torch.cat(v) for v in ys], graph


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--sequences", type=int, default=4)
    p.add_argument("--prompt", type=int, default=200)
    p.add_argument("--steps", type=int, default=8)
    a = p.parse_args()
    prompts = [max(1, a.prompt - 37 * s) for s in range(a.sequences)]
    pages = a.sequences * ((a.prompt + a.steps + 15) // 16)
    layer = Layer(a.hidden, a.heads, pages=pages)
    xs, ys, graph = serve(layer, prompts, a.steps)
    want = layer.plain(torch.cat(xs), [len(v) for v in xs])
    error = float((torch.cat(ys).float() - want).norm() / want.norm())
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{sum(prompts)} prompt tokens and {a.steps} x {a.sequences} decoded ones; against a plain float32 layer without "
          f"a cache: {error:.2e} (the 8-bit cache's part); one decoding step {begin.elapsed_time(end) / 20 * 1e3:.0f} us")


if __name__ == "__main__":
    main()
