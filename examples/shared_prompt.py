"""A batch that shares its prompt, through a small hybrid model.

Three KDA layers and a softmax-attention layer with random weights.  The prompt is
run once: its KDA states are the start of every sequence, its keys and values lie
in the cache once.  Then every sequence decodes for itself, with the calls in the
places where a serving loop has them:

    kda_prefill, kda_decode_step    the KDA layers, prompt and steps
    kda_head_norm_rope              the softmax layer's queries and keys
    kda_prefix_attention            the softmax layer, over the shared prompt and each sequence's own pages
    kda_cache_append                new keys and values into the pages
    kda_sample                      the next tokens, with each sequence's own settings

    python examples/shared_prompt.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_03_gb300 import kda  # noqa: E402

H, D = 2, 128                       # KDA heads
HQ, HKV, DA = 8, 2, 64              # softmax heads
HIDDEN, VOCAB, PAGE = 256, 1009, 16


class Hybrid:
    """The model's weights; the states, pages and lengths of `n` sequences behind one prompt."""

    def __init__(self, n, max_prompt=512, max_new=64, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        w = lambda i, o, s=1.0: (torch.randn(i, o, generator=gen, device=device) * s * i ** -0.5).bfloat16()
        self.embed = torch.randn(VOCAB, HIDDEN, generator=gen, device=device).bfloat16()
        self.kda = [dict(q=w(HIDDEN, H * D), k=w(HIDDEN, H * D), v=w(HIDDEN, H * D), g=w(HIDDEN, H * D),
                         b=w(HIDDEN, H), o=w(H * D, HIDDEN)) for _ in range(3)]
        # queries, keys and values side by side, out of one product
        self.qkv, self.o = w(HIDDEN, (HQ + 2 * HKV) * DA), w(HQ * DA, HIDDEN)
        self.q_norm, self.k_norm = (1 + 0.1 * torch.randn(DA, generator=gen, device=device) for _ in range(2))
        self.inv_freq = 10000.0 ** (-torch.arange(DA // 2, device=device) / (DA // 2))
        self.head = w(HIDDEN, VOCAB, 2.0)
        self.n, self.device = n, device
        shared, own = -(-max_prompt // PAGE), -(-max_new // PAGE)
        pages = torch.randperm(shared + n * own, generator=gen, device=device).int()
        self.prefix_table, self.table = pages[None, :shared].contiguous(), pages[shared:].view(n, own)
        self.k_cache = torch.zeros(len(pages), HKV, PAGE, DA, device=device, dtype=torch.bfloat16)
        self.v_cache = torch.zeros_like(self.k_cache)
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=device)
        self.prefix_lens, self.prefix_seqs = i32(0), i32(0, n)
        self.lens = torch.zeros(n, dtype=torch.int32, device=device)
        self.root = torch.full((n, 1), -1, dtype=torch.int32, device=device)
        self.state = None
        self.workspace = torch.zeros(kda.kda_prefix_attention_workspace_size(
            HQ, HKV, DA, torch.bfloat16, n, 1, 1, PAGE, shared, own), dtype=torch.uint8, device=device)

    @staticmethod
    def _norm(x):
        x = x.float()
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def _kda_inputs(self, layer, x):
        y = self._norm(x).bfloat16()
        heads = lambda name: (y @ layer[name]).view(-1, H, D)
        unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).bfloat16()
        g = -5 * torch.sigmoid(heads("g").float() - 2)
        return unit(heads("q")), unit(heads("k")), heads("v").contiguous(), g, torch.sigmoid((y @ layer["b"]).float()).contiguous()

    def _softmax_inputs(self, x, positions):
        qkv = (self._norm(x).bfloat16() @ self.qkv).view(-1, HQ + 2 * HKV, DA)
        q, k = kda.kda_head_norm_rope(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], positions, self.inv_freq, self.q_norm, self.k_norm)
        return q, k, qkv[:, HQ + HKV:].contiguous()

    def _logits(self, x):
        return (self._norm(x).bfloat16() @ self.head).float()

    def prompt(self, tokens):
        """The prompt's tokens [T], run once for all; the logits after the last one, for every sequence.

        The prompt's softmax attention goes through the tree call, 64 tokens at a time."""
        T = len(tokens)
        x = self.embed[tokens.long()].float()
        self.state = []
        for layer in self.kda:
            q, k, v, g, beta = self._kda_inputs(layer, x)
            out, state = kda.kda_prefill(q, k, v, g, beta)
            x = x + (out.view(T, H * D) @ layer["o"]).float()
            self.state.append(state.expand(self.n, -1, -1, -1).contiguous())
        q, k, v = self._softmax_inputs(x, torch.arange(T, dtype=torch.int32, device=self.device))
        lens, parts = torch.zeros(1, dtype=torch.int32, device=self.device), []
        for t in range(0, T, 64):
            rows = slice(t, min(t + 64, T))
            chain = torch.arange(rows.stop - t, dtype=torch.int32, device=self.device)[None] - 1
            part, _ = kda.kda_tree_attention(q[rows], k[rows], v[rows], self.k_cache, self.v_cache, self.prefix_table, lens,
                                             chain)
            parts.append(part)
            lens = kda.kda_cache_append(k[rows], v[rows], self.k_cache, self.v_cache, self.prefix_table, lens)
        self.prefix_lens = lens
        x = x + (torch.cat(parts).view(T, HQ * DA) @ self.o).float()
        return self._logits(x[-1:]).expand(self.n, -1).contiguous()

    def step(self, tokens):
        """One token per sequence; the logits [n, VOCAB] after it."""
        n = self.n
        x = self.embed[tokens.long()].float()
        for layer, state in zip(self.kda, self.state):
            out = kda.kda_decode_step(*self._kda_inputs(layer, x), state)
            x = x + (out.view(n, H * D) @ layer["o"]).float()
        q, k, v = self._softmax_inputs(x, self.prefix_lens + self.lens)
        out, _ = kda.kda_prefix_attention(q, k, v, self.k_cache, self.v_cache, self.prefix_table, self.prefix_lens,
                                          self.prefix_seqs, self.table, self.lens, self.root, workspace=self.workspace)
        self.lens = kda.kda_cache_append(k, v, self.k_cache, self.v_cache, self.table, self.lens)
        return self._logits(x + (out.view(n, HQ * DA) @ self.o).float())

    def check(self):
        """Raises what the last attention call found (waits for the GPU)."""
        if kda.kda_get_device_status(self.workspace) != kda.KDA_DEVICE_OK:
            raise kda.KDAError(kda.KDA_ERR_DEVICE, "kda_prefix_attention")


def generate(model, prompt, steps, seed=0, **settings):
    """`steps` tokens for every sequence; settings as kda_sample's.  Returns [n, steps] int32."""
    gen = torch.Generator(device=model.device).manual_seed(seed)
    logits, out = model.prompt(prompt), []
    for _ in range(steps):
        token, _ = kda.kda_sample(logits, torch.rand(model.n, generator=gen, device=model.device), **settings)
        out.append(token)
        logits = model.step(token)
    model.check()
    return torch.stack(out, 1)


def main():
    model = Hybrid(n=6, seed=1)
    prompt = torch.randint(0, VOCAB, (200,), generator=torch.Generator().manual_seed(2)).cuda()
    per = lambda *x: torch.tensor(x, device="cuda")
    tokens = generate(model, prompt, steps=12, seed=3, temperature=per(0.0, 0.7, 0.7, 1.0, 1.0, 1.2),
                      top_k=per(0, 20, 0, 50, 0, 0).int(), top_p=per(1.0, 1.0, 0.9, 0.95, 1.0, 0.8))
    for row in tokens.tolist():
        print(row)


if __name__ == "__main__":
    main()
