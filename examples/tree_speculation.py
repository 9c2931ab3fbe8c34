"""Decoding with trees of drafted tokens through a small hybrid model.

Three KDA layers and a softmax-attention layer with random weights, a batch of
sequences, and the five tree calls in the places where a serving loop has them:

    kda_decode_tree      every KDA layer, all drafted nodes from the read-only state
    kda_tree_attention   the softmax layer, over its paged cache and the tree
    kda_verify_drafts    the kept path and the next token
    kda_decode_commit    the KDA states behind the kept path
    kda_cache_append     the kept path's keys and values into the pages

The drafts are the likeliest successors under a table (the model's own output
for each token alone), a poor draft that still gets some tokens kept.  The
prompt goes through the same calls, as a chain that is kept whole.

    python examples/tree_speculation.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_03_gb300 import kda  # noqa: E402

H, D = 2, 128                       # KDA heads
HQ, HKV, DA = 4, 2, 64              # softmax heads
HIDDEN, VOCAB, PAGE = 256, 101, 16


class Hybrid:
    """The model's weights, and the states and pages of `n` sequences."""

    def __init__(self, n, max_tokens=256, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        w = lambda i, o, s=1.0: (torch.randn(i, o, generator=gen, device=device) * s * i ** -0.5).bfloat16()
        self.embed = torch.randn(VOCAB, HIDDEN, generator=gen, device=device).bfloat16()
        self.kda = [dict(q=w(HIDDEN, H * D), k=w(HIDDEN, H * D), v=w(HIDDEN, H * D), g=w(HIDDEN, H * D),
                         b=w(HIDDEN, H), o=w(H * D, HIDDEN)) for _ in range(3)]
        self.att = dict(q=w(HIDDEN, HQ * DA, 2.0), k=w(HIDDEN, HKV * DA), v=w(HIDDEN, HKV * DA), o=w(HQ * DA, HIDDEN))
        self.head = w(HIDDEN, VOCAB, 2.0)
        self.n, self.device = n, device
        self.state = [torch.zeros(n, H, D, D, device=device) for _ in self.kda]
        per = -(-max_tokens // PAGE)
        self.table = torch.randperm(n * per, generator=gen, device=device).int().view(n, per)
        self.k_cache = torch.zeros(n * per, HKV, PAGE, DA, device=device, dtype=torch.bfloat16)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.lens = torch.zeros(n, dtype=torch.int32, device=device)
        self.workspaces = {}                # by nodes per sequence

    def workspace(self, M):
        """The attention's workspace, kept: its status word tells of pages and lengths out of range."""
        if M not in self.workspaces:
            size = kda.kda_tree_attention_workspace_size(HQ, HKV, DA, torch.bfloat16, self.n, M, PAGE,
                                                         self.table.shape[1])
            self.workspaces[M] = torch.zeros(size, dtype=torch.uint8, device=self.device)
        return self.workspaces[M]

    def check(self):
        """Raises what the last attention call with each workspace found (waits for the GPU)."""
        for ws in self.workspaces.values():
            if kda.kda_get_device_status(ws) != kda.KDA_DEVICE_OK:
                raise kda.KDAError(kda.KDA_ERR_DEVICE, "kda_tree_attention")

    @staticmethod
    def _norm(x):
        x = x.float()
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def forward(self, tokens, parent):
        """Probabilities [n, M, VOCAB] after every node, and what a commit needs."""
        n, M = tokens.shape
        x = self.embed[tokens.long().clamp(0, VOCAB - 1)].view(n * M, HIDDEN).float()
        kept = []
        for layer, state in zip(self.kda, self.state):
            y = self._norm(x).bfloat16()
            heads = lambda name: (y @ layer[name]).view(n * M, H, D)
            unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).bfloat16()
            q, k, v = unit(heads("q")), unit(heads("k")), heads("v").contiguous()
            g = -5 * torch.sigmoid(heads("g").float() - 2)
            beta = torch.sigmoid((y @ layer["b"]).float()).contiguous()
            out = kda.kda_decode_tree(q, k, v, g, beta, state, parent)
            x = x + (out.view(n * M, H * D) @ layer["o"]).float()
            kept.append((k, v, g, beta))
        y = self._norm(x).bfloat16()
        q = (y @ self.att["q"]).view(n * M, HQ, DA)
        k, v = ((y @ self.att[c]).view(n * M, HKV, DA) for c in "kv")
        out, _ = kda.kda_tree_attention(q, k, v, self.k_cache, self.v_cache, self.table, self.lens, parent,
                                        workspace=self.workspace(M))
        x = x + (out.view(n * M, HQ * DA) @ self.att["o"]).float()
        kept.append((k, v))
        logits = (self._norm(x).bfloat16() @ self.head).float()
        return torch.softmax(logits, -1).view(n, M, VOCAB), kept

    def commit(self, kept, path, accept):
        """States and pages behind the first accept[n] nodes of path[n]."""
        for (k, v, g, beta), state in zip(kept, self.state):
            kda.kda_decode_commit(k, v, g, beta, state, path, accept)
        k, v = kept[-1]
        self.lens = kda.kda_cache_append(k, v, self.k_cache, self.v_cache, self.table, self.lens, path=path,
                                         accept=accept)

    def feed(self, tokens):
        """tokens [n, T] (T <= 64) kept whole; the distribution after the last."""
        n, T = tokens.shape
        chain = torch.arange(T, dtype=torch.int32, device=self.device).expand(n, T).contiguous()
        probs, kept = self.forward(tokens, chain - 1)
        self.commit(kept, chain, torch.full((n,), T, dtype=torch.int32, device=self.device))
        return probs[:, -1]


def successors(model, width):
    """[VOCAB, width]: a table of likely next tokens, from the head alone."""
    logits = model._norm(model.embed).bfloat16() @ model.head
    return logits.float().topk(width, -1).indices.int()


def draft(table, last, shape):
    """A tree below `last`: node m is its parent's shape[m][1]-th successor."""
    tokens = [last]
    for parent, rank in shape[1:]:
        tokens.append(table[tokens[parent].long(), rank])
    parent = torch.tensor([p for p, _ in shape], dtype=torch.int32, device=last.device)
    return torch.stack(tokens, 1).int().contiguous(), parent.expand(len(last), -1).contiguous()


# (parent, rank among its successors): three below the root, two and one below the first of those, ...
SHAPE = [(-1, 0), (0, 0), (0, 1), (0, 2), (1, 0), (1, 1), (2, 0), (4, 0), (4, 1), (7, 0)]


def generate(model, prompt, steps, seed=0):
    """`steps` tree steps after the prompt [n, T]; the token lists and the mean kept path."""
    gen = torch.Generator(device=model.device).manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=gen, device=model.device)
    n, M = len(prompt), len(SHAPE)
    table = successors(model, 3)
    probs = model.feed(prompt)
    # the first token comes from the prompt's last distribution alone (a tree of one node)
    root = torch.full((n, 1), -1, dtype=torch.int32, device=model.device)
    _, _, last = kda.kda_verify_drafts(probs.view(n, 1, VOCAB).contiguous(), prompt[:, -1:].int().contiguous(), root,
                                       rand(n, 2))
    out, kept_nodes = [prompt[i].tolist() for i in range(n)], 0
    for _ in range(steps):
        tokens, parent = draft(table, last, SHAPE)
        probs, kept = model.forward(tokens, parent)
        accept, path, last = kda.kda_verify_drafts(probs, tokens, parent, rand(n, M + 1))
        model.commit(kept, path, accept)
        for i, (a, row) in enumerate(zip(accept.tolist(), path.tolist())):
            out[i] += [int(tokens[i, m]) for m in row[:a]]
            kept_nodes += a
    model.check()
    return [o + [int(t)] for o, t in zip(out, last.tolist())], kept_nodes / (n * steps)


def main():
    model = Hybrid(n=4, seed=1)
    prompt = torch.randint(0, VOCAB, (4, 12), generator=torch.Generator().manual_seed(2)).int().cuda()
    tokens, mean = generate(model, prompt, steps=12, seed=3)
    for t in tokens:
        print(len(t), t)
    print(f"{mean:.2f} tokens kept per step")


if __name__ == "__main__":
    main()
