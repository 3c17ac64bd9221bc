"""One attention block of a quantized model, prompt and single tokens, on the package's calls:

    x -> quantize_act -> q, k (one fused q4_K weight), v (q6_K) -> rotary positions
      -> kv_write -> kv_attend -> quantize_act -> output product (q4_K) -> x + y

The cache is paged and holds 4.5 bits a value.  Random weights and inputs; the block runs a
batch's prompts, then one token per sequence and step, and checks the steps against the same
rows computed as one prompt.

    python examples/attention_block.py --prompt 300 --steps 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quant_int8_mmq_gb300 as mmq  # noqa: E402
import synth  # noqa: E402

DEV = "cuda"


def rotate(x, pos):
    """Rotary positions: x [tokens, heads, dim], pos [tokens]."""
    half = x.shape[-1] // 2
    freq = 10000.0 ** (-torch.arange(half, device=x.device) / half)
    angle = pos[:, None, None] * freq
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)


class Block:
    def __init__(self, hidden, heads, kv_heads, dim, seed=0):
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim

        def raw(kind, rows, cols, s):
            return torch.from_numpy(synth.blocks(kind, rows, cols, seed + s).reshape(-1)).to(DEV)

        nq, nk = heads * dim, kv_heads * dim
        self.qk = mmq.pack_weights_fused("q4_K", raw("q4_K", nq, hidden, 1), nq, raw("q4_K", nk, hidden, 2), nk, hidden)
        self.v = mmq.pack_weights("q6_K", raw("q6_K", nk, hidden, 3), nk, hidden)
        self.o = mmq.pack_weights("q4_K", raw("q4_K", hidden, nq, 4), hidden, nq)

    def __call__(self, x, cache, max_q, max_kv):
        """x [tokens, hidden] f32, the newest tokens of each sequence of the cache
        (pages, table, start, length); length counts them already."""
        n, nq, nk = x.shape[0], self.heads * self.dim, self.kv_heads * self.dim
        pages, table, start, length = cache
        qa, sc = mmq.quantize_act(x)
        qk = mmq.gemm("q4_K", self.qk, nq + nk, self.hidden, qa, sc, n)
        v = mmq.gemm("q6_K", self.v, nk, self.hidden, qa, sc, n)
        seq = torch.searchsorted(start[1:], torch.arange(n, device=DEV, dtype=torch.int32), right=True)
        pos = length[seq] - start[seq + 1] + torch.arange(n, device=DEV)
        # random weights give rows of any size; a model's training keeps them near 1
        q = rotate(torch.nn.functional.normalize(qk[:, :nq].view(n, self.heads, self.dim), dim=-1) * self.dim ** 0.5, pos)
        k = rotate(torch.nn.functional.normalize(qk[:, nq:].view(n, self.kv_heads, self.dim), dim=-1) * self.dim ** 0.5,
                   pos)
        mmq.kv_write(k, v.view(n, self.kv_heads, self.dim), *cache)
        out = mmq.kv_attend(q, *cache, max_q=max_q, max_kv=max_kv)
        qa, sc = mmq.quantize_act(out.view(n, nq))
        return out, x + mmq.gemm("q4_K", self.o, self.hidden, nq, qa, sc, n)


def tables(lengths, spare=0):
    """A page table for sequences of up to these lengths, its pages in no order."""
    need = [-(-m // mmq.KV_PAGE) for m in lengths]
    perm = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.to(DEV), sum(need) + spare


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128, choices=(64, 128))
    ap.add_argument("--prompt", type=int, default=300, help="longest prompt of the batch")
    ap.add_argument("--batch", type=int, default=3)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args(argv)
    block = Block(a.hidden, a.heads, a.kv_heads, a.dim)
    prompts = [max(1, a.prompt * (a.batch - b) // a.batch) for b in range(a.batch)]
    total = [n + a.steps for n in prompts]
    gen = torch.Generator(DEV).manual_seed(2)
    xs = [torch.randn(n, a.hidden, device=DEV, generator=gen) for n in total]
    table, num = tables(total)

    def cumulative(counts):
        return ints([sum(counts[:i]) for i in range(len(counts) + 1)])

    # the prompts at once, then a token of each sequence a step
    pages = mmq.kv_pages(num, a.kv_heads, a.dim, device=DEV)
    length = ints(prompts)
    block(torch.cat([x[:n] for x, n in zip(xs, prompts)]), (pages, table, cumulative(prompts), length), max(prompts),
          max(prompts))
    one = cumulative([1] * a.batch)
    got = []
    for s in range(a.steps):
        length += 1
        got.append(block(torch.stack([x[n + s] for x, n in zip(xs, prompts)]), (pages, table, one, length), 1, max(total))[0])

    # the same rows as one prompt, on a cache of its own
    pages = mmq.kv_pages(num, a.kv_heads, a.dim, device=DEV)
    want, _ = block(torch.cat(xs), (pages, table, cumulative(total), ints(total)), max(total), max(total))
    st = mmq.mmq_get_device_error()
    if st:
        raise RuntimeError(mmq.mmq_status_string(st))
    worst = 0.0
    for b, n in enumerate(prompts):
        rows = want[sum(total[:b]) + n:sum(total[:b + 1])]
        steps = torch.stack([g[b] for g in got])
        worst = max(worst, ((steps - rows).norm() / rows.norm()).item())
    print(f"{a.batch} prompts of up to {max(prompts)} tokens, {a.steps} steps: steps and prompt differ by {worst:.1e}")
    return worst


if __name__ == "__main__":
    main()
