"""Speculative decoding of a small random model on one GPU, every step of it through the library.

    python examples/speculative.py [--mode chain|tree|plain] [--temperature T] [--rounds N]
                                     [--top-k K] [--top-p P] [--min-p P]

A two-layer decoder with MXFP8 key/value caches and e4m3 twin weights. The drafter is the same model left after its
first layer, so both share that layer's cache. A round drafts a chain of five tokens (or a tree of seven nodes: two
guesses after the root and after each of them), runs root and drafts through the whole model in one pass, verifies them
against the target's logits, and keeps what was accepted: a tree's accepted nodes are moved to the sequence's end by
reading their cache rows and writing them back, which reproduces codes and scales bit for bit. Nothing waits for the GPU
inside a round. At temperature 0 the tokens are those of plain decoding. Rules (top-k, top-p, min-p) filter drafts' and
target's logits alike, so what stands is distributed as the filtered target.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_skinny_amd as L  # noqa: E402

VOCAB, WIDTH, LAYERS, HQ, HKV, DIM, PAGE = 2048, 512, 2, 8, 2, 64, 16


class Model:
    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.device = device

        def twin(n, k):                                  # e4m3 codes of unit variance times a power of two near k^-1/2
            q = torch.randn(1, n, k, generator=g, device=device).to(torch.float8_e4m3fn).view(torch.uint8)
            e = torch.full((1, n // 32, k // 32), 127 - (k.bit_length() - 1) // 2, dtype=torch.uint8, device=device)
            return q, e

        self.embed = torch.randn(VOCAB, WIDTH, generator=g, device=device).to(torch.bfloat16)
        self.qkv = [twin((HQ + 2 * HKV) * DIM, WIDTH) for _ in range(LAYERS)]
        self.o = [twin(WIDTH, HQ * DIM) for _ in range(LAYERS)]
        self.head = twin(VOCAB, WIDTH)
        self.weight = torch.ones(DIM, dtype=torch.bfloat16, device=device)
        a = torch.arange(4096, device=device, dtype=torch.float64)[:, None]
        a = a * 10000.0 ** (-torch.arange(DIM // 2, device=device, dtype=torch.float64) / (DIM // 2))
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float()

    def forward(self, caches, pages, tokens, lens, positions, mask=None, layers=LAYERS):
        """Logits fp32 [B, T, VOCAB] of tokens int32 [B, T] that follow the lens tokens of each sequence; their keys and
        values enter the first `layers` caches."""
        B, T = tokens.shape
        at = lens[:, None].long() + torch.arange(T, device=self.device)
        slots = slots_of(pages, at).flatten()
        held = lens + T
        h = self.embed[tokens.flatten().long()]
        for i in range(layers):
            qkv = L.bsfp8_gemm(norm(h), *self.qkv[i]).squeeze(1)
            q, k, v = qkv.split([HQ * DIM, HKV * DIM, HKV * DIM], 1)
            q = L.bsfp8_cache_write(caches[i], slots, k, v, q=q, q_weight=self.weight, k_weight=self.weight,
                                    cos_sin=self.cos_sin, positions=positions.flatten())
            y = L.bsfp8_tree_attention(q.view(B, T, HQ, DIM), caches[i], pages, held, mask=mask)
            h = h + L.bsfp8_gemm(y.view(B * T, HQ * DIM), *self.o[i]).squeeze(1)
        return L.bsfp8_gemm(norm(h), *self.head, out_dtype="f32").view(B, T, VOCAB)


def norm(h):
    x = h.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def slots_of(pages, at):
    """Slots of positions at [B, T] (-1 where at is negative)."""
    pg = pages.gather(1, (at.clamp(min=0) // PAGE)).long()
    return torch.where(at >= 0, pg * PAGE + at % PAGE, -1)


# a tree of seven nodes: its parents, depths, and each node's mask of ancestors and itself
PARENTS, DEPTH = [-1, 0, 0, 1, 1, 2, 2], [0, 1, 1, 2, 2, 2, 2]
MASKS = [1 << i | (1 << p | 1 if p >= 0 else 0) for i, p in enumerate(PARENTS)]


def generate(model, prompt, rounds, mode="chain", temperature=0.0, seed=0, drafts=5, top_k=0, top_p=1.0, min_p=0.0):
    """prompt int32 [B, P] -> the tokens that each sequence generated in `rounds` rounds, and how many drafts a round
    were accepted on the average."""
    dev, (B, P) = model.device, prompt.shape
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    T = {"plain": 1, "chain": drafts + 1, "tree": len(PARENTS)}[mode]
    width = (P + (rounds + 1) * T + PAGE - 1) // PAGE
    caches = [L.KVCache.empty(B * width, HKV, PAGE, DIM, device=dev) for _ in range(LAYERS)]
    pages = torch.randperm(B * width, generator=g, device=dev).view(B, width).to(torch.int32)
    t = torch.full((B,), float(temperature), device=dev)
    rand = lambda *s: torch.rand(*s, generator=g, device=dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev).expand(B, -1).contiguous()

    rules = temperature > 0 and (top_k > 0 or top_p < 1 or min_p > 0)

    def sample(logits):                                  # [B, n, VOCAB], filtered by the rules -> int32 [B, n]
        if rules:
            R = logits.shape[0] * logits.shape[1]
            every = lambda x, dtype: torch.full((R,), x, dtype=dtype, device=dev)
            rows = logits.view(R, VOCAB)
            return L.bsfp8_sample(rows, every(temperature, torch.float32), rand(R), every(top_k, torch.int32),
                                  every(top_p, torch.float32), every(min_p, torch.float32), filtered=rows).view(logits.shape[:2])
        if temperature == 0:
            return logits.argmax(-1).to(torch.int32)
        p = torch.softmax(logits / temperature, -1)
        return torch.multinomial(p.flatten(0, 1), 1, generator=g).view(p.shape[:2]).to(torch.int32)

    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    logits = model.forward(caches, pages, prompt, lens, torch.arange(P, device=dev).expand(B, P))
    lens = lens + P
    out, accepted = [sample(logits[:, -1:].contiguous())], []
    root = out[0]
    ws = L.workspace_verify(B, T, VOCAB, device=dev)
    parents, masks = i32(PARENTS), torch.tensor(MASKS, device=dev).expand(B, -1).contiguous()
    depth = torch.tensor(DEPTH, device=dev)
    row = torch.arange(T, device=dev)
    for _ in range(rounds):
        first = lens[:, None].long()
        if mode == "tree":
            tokens = root
            for level in (1, 3):                         # two guesses after each node of the last level
                n = tokens.shape[1]
                lg = model.forward(caches, pages, tokens, lens, first + depth[:n], mask=masks[:, :n].contiguous(), layers=1)
                best = lg[:, n // 2:].topk(2, -1).indices.flatten(1)
                tokens = torch.cat([tokens, best.to(torch.int32)], 1)
            logits = model.forward(caches, pages, tokens, lens, first + depth, mask=masks)
            if rules:
                sample(logits)
            got, path, n = L.bsfp8_verify_tree(logits, tokens, parents, t, rand(B, T), ws=ws)
            # the accepted nodes' rows, one after another from the sequence's end
            src = slots_of(pages, torch.where(path >= 0, first + path, -1)).flatten()
            dst = slots_of(pages, torch.where(path >= 0, first + row, -1)).flatten()
            for c in caches:
                L.bsfp8_cache_write(c, dst, *L.bsfp8_cache_read(c, src))
        else:
            tokens, draft = [root], []
            for i in range(T - 1):
                draft.append(model.forward(caches, pages, tokens[-1], lens + i, first + i, layers=1))
                tokens.append(sample(draft[-1]))
            draft = torch.cat(draft, 1) if draft else torch.empty(B, 0, VOCAB, device=dev)
            tokens = torch.cat(tokens, 1)
            logits = model.forward(caches, pages, tokens, lens, first + row)
            if rules:
                sample(logits)
            got, n = L.bsfp8_verify_chain(logits, draft, tokens[:, 1:].contiguous(), t, rand(B, T - 1), rand(B), ws=ws)
        lens = lens + n + 1
        root = got.gather(1, n[:, None].long())
        out.append(got)
        accepted.append(n)
    out = torch.cat(out, 1).cpu()
    return [[x for x in s if x >= 0] for s in out.tolist()], torch.stack(accepted).float().mean().item()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--mode", choices=("plain", "chain", "tree"), default="chain")
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--top-k", type=int, default=0, help="0: all")
    ap.add_argument("--top-p", type=float, default=1.0, help="1: all")
    ap.add_argument("--min-p", type=float, default=0.0, help="0: all")
    ap.add_argument("--rounds", type=int, default=24, help="each gives at least one token a sequence")
    a = ap.parse_args()
    model = Model()
    prompt = torch.randint(0, VOCAB, (2, 12), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    text, mean = generate(model, prompt, a.rounds, a.mode, a.temperature, top_k=a.top_k, top_p=a.top_p, min_p=a.min_p)
    for s in text:
        print(s)
    print(f"{mean:.2f} drafts accepted a round")


if __name__ == "__main__":
    main()
