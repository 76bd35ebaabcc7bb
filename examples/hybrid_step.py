"""A hybrid model's token mixing over one pool of pages: a recurrent (KDA) layer, a layer that
attends over an 8-bit cache, and one that attends over a 16-bit cache through a sliding window.

Ragged prompts are prefilled, then every sequence decodes a token at a time from one captured CUDA
graph.  The same tokens prefilled in one go have to give the same answers, which is checked.

    python examples/hybrid_step.py
"""
import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import numpy as np
import torch

import kda_state_chunked_gb300 as kda

BF16 = torch.bfloat16


def _weight(gen, n_out, n_in, device):
    return (torch.randn(n_in, n_out, generator=gen) * n_in ** -0.5).to(device, BF16)


def _norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.pow(2).mean(-1, keepdim=True) + 1e-6)).to(BF16)


class Batch:
    """One call's tokens: nseq sequences with n[s] new tokens behind start[s] earlier ones."""

    def __init__(self, n, start, device):
        self.n, self.start = np.asarray(n, np.int32), np.asarray(start, np.int64)
        self.cu = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.max_q = int(self.n.max())
        self.cu_dev = torch.from_numpy(self.cu).to(device)
        self.len_dev = torch.from_numpy((self.start + self.n).astype(np.int32)).to(device)


class KdaLayer:
    """q, k, v and the two gates of each token from one projection; the state is a page object."""

    def __init__(self, gen, pool, width, H, d, nseq, device):
        self.pool, self.H, self.d, self.nseq = pool, H, d, nseq
        self.w_in = _weight(gen, 4 * H * d + H, width, device)
        self.w_out = _weight(gen, width, H * d, device)
        self.conv = (torch.randn(H, 3 * d, 4, generator=gen) * 0.5).to(device)
        self.new_cache()

    def new_cache(self):
        P = self.pool.object_pages(self.H, self.d, kda.KDA_BF16)
        self.pages = kda.kda_page_alloc(self.pool, self.nseq * P).reshape(self.nseq, P)
        self.pages_dev = torch.from_numpy(self.pages).to(self.w_in.device)

    def __call__(self, x, b, status):
        T, H, d = x.shape[0], self.H, self.d
        y = _norm(x) @ self.w_in
        q, k, v, a = (t.reshape(T, H, d) for t in y[:, :4 * H * d].chunk(4, dim=1))
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(BF16) for t in (q, k))
        a = (0.95 + 0.05 * torch.sigmoid(a.float())).to(BF16)       # forget gate
        beta = torch.sigmoid(y[:, 4 * H * d:]).contiguous()
        o = torch.empty(T, H, d, dtype=BF16, device=x.device)
        if (b.n == 1).all() and b.start.min() > 0:
            kda.kda_decode_step(self.pool, q, k, v.contiguous(), a, beta, self.conv, o, self.pages_dev, status)
        else:
            ws = kda.prefill_workspace(q, b.cu, b.start, 0, self.pages.shape[1])
            kda.kda_prefill_varlen(self.pool, b.cu, b.start, b.start > 0, q, k, v.contiguous(), a, beta, self.conv, o,
                                   self.pages, workspace=ws, status=status)
        return x + o.reshape(T, H * d) @ self.w_out


class AttnLayer:
    """Attention over a paged cache; pages are taken for the longest a sequence may become."""

    def __init__(self, gen, pool, width, Hq, Hkv, d, fmt, page_tokens, nseq, max_len, cos_sin, device, window=0,
                 sinks=0):
        self.pool, self.Hq, self.Hkv, self.d, self.nseq = pool, Hq, Hkv, d, nseq
        self.fmt, self.pt, self.window, self.sinks, self.cos_sin = fmt, page_tokens, window, sinks, cos_sin
        self.w_in = _weight(gen, (Hq + 2 * Hkv) * d, width, device)
        self.w_out = _weight(gen, width, Hq * d, device)
        self.blocks = -(-max_len // page_tokens)
        self.ws = {}
        self.new_cache()

    def new_cache(self):
        ids = kda.kda_page_alloc(self.pool, self.nseq * self.blocks).reshape(self.nseq, self.blocks)
        self.table = torch.from_numpy(ids).to(self.w_in.device)

    def __call__(self, x, b, status):
        T, Hq, Hkv, d = x.shape[0], self.Hq, self.Hkv, self.d
        y = (_norm(x) @ self.w_in).view(T, Hq + 2 * Hkv, d)         # the calls take its parts as they lie
        q, k, v = y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]
        turned = torch.empty(T, Hq, d, dtype=BF16, device=x.device)
        kda.kda_kv_append(self.pool, self.fmt, self.pt, b.cu_dev, b.len_dev, self.table, b.max_q, q, k, v, self.cos_sin,
                          turned, status)
        if (T, b.max_q) not in self.ws:
            self.ws[T, b.max_q] = kda.attn_workspace(turned, Hkv, self.nseq, b.max_q)
        o = torch.empty_like(turned)
        kda.kda_attn_paged(self.pool, Hkv, self.fmt, self.pt, b.cu_dev, b.len_dev, self.table, b.max_q, turned, o,
                           self.ws[T, b.max_q], status, window=self.window, sinks=self.sinks)
        return x + o.view(T, Hq * d) @ self.w_out


def run(prompts=(700, 1, 129, 64), steps=8, width=512, Hq=16, Hkv=4, d=128, window=96, sinks=4, device="cuda"):
    """Prefill and decode, then prefill alone.  Returns (difference of the two, relative to the
    answers' root mean square, ms of the prompts' prefill, ms of a decode step)."""
    gen = torch.Generator().manual_seed(5)
    nseq, max_len, pt = len(prompts), max(prompts) + steps, 64
    # one page size serves all: the larger of the two caches' blocks
    page = max(kda.kda_kv_page_bytes(Hkv, d, f, pt) for f in (kda.KDA_KV_I8, kda.KDA_KV_BF16))
    states = -(-kda.kda_object_bytes(Hq, d, kda.KDA_BF16) // page)
    pool = kda.Pool(page, 2 * nseq * (states + 2 * -(-max_len // pt)), device)
    status = torch.zeros(1, dtype=torch.int32, device=device)
    # rotation table: a row's cosines, then its sines
    ang = torch.arange(max_len)[:, None] * 10000.0 ** (-torch.arange(0, d, 2) / d)
    cos_sin = torch.cat([ang.cos(), ang.sin()], dim=1).float().to(device)
    attn = (gen, pool, width, Hq, Hkv, d)
    layers = [KdaLayer(gen, pool, width, Hq, d, nseq, device),
              AttnLayer(*attn, kda.KDA_KV_I8, pt, nseq, max_len, cos_sin, device),
              AttnLayer(*attn, kda.KDA_KV_BF16, pt, nseq, max_len, cos_sin, device, window, sinks)]
    xs = [torch.randn(n + steps, width, generator=gen).to(device, BF16) for n in prompts]

    def forward(x, b):
        for layer in layers:
            x = layer(x, b, status)
        return x

    ev = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    first = Batch(prompts, [0] * nseq, device)
    x = torch.cat([x[:n] for x, n in zip(xs, prompts)])
    ev[0].record()
    forward(x, first)
    ev[1].record()

    # Decode: the graph holds one step, and the lengths on the device that it starts by raising.
    b = Batch([1] * nseq, prompts, device)
    b.len_dev -= 1
    x_in = torch.zeros(nseq, width, dtype=BF16, device=device)

    def step():
        b.len_dev.add_(1)
        return forward(x_in, b)

    def tokens(i):
        return torch.stack([x[n + i] for x, n in zip(xs, prompts)])

    outs = []
    x_in.copy_(tokens(0))
    side = torch.cuda.Stream(device)                # the first step runs eagerly and warms the graph's calls up
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs.append(step().clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    ev[2].record()
    for i in range(1, steps):
        x_in.copy_(tokens(i))
        graph.replay()
        outs.append(y.clone())
    ev[3].record()
    decoded = torch.stack(outs, dim=1)              # [nseq, steps, width]

    for layer in layers:                            # all tokens at once, into new pages
        layer.new_cache()
    whole = forward(torch.cat(xs), Batch([n + steps for n in prompts], [0] * nseq, device))
    ends = np.cumsum([n + steps for n in prompts])
    wanted = torch.stack([whole[e - steps:e] for e in ends])
    code, bits = kda.kda_sync_status(status)
    if code != kda.KDA_OK:
        raise RuntimeError(f"device status bits {bits:#x}")
    added = wanted.double() - torch.stack([x[n:] for x, n in zip(xs, prompts)]).double()   # what the layers add
    diff = (decoded.double() - wanted.double()).pow(2).mean().sqrt() / added.pow(2).mean().sqrt()
    pool.close()
    return float(diff), ev[0].elapsed_time(ev[1]), ev[2].elapsed_time(ev[3]) / max(1, steps - 1)


# The two ways round keys, values and states at other places.  An 8-bit block that grew a token at a
# time has been coded anew each time its maximum rose: a step of max / 127, some 0.03 of the values'
# size, whose rounding (0.03 / sqrt 12) counts twice or three times over on either side, in keys and
# in values: 0.03 at most.  bf16 roundings (0.004 each, a dozen on the way) add 0.015.
BOUND = 0.05

if __name__ == "__main__":
    run()                                           # first calls load the kernels
    diff, prefill_ms, step_ms = run()
    print(f"prompts {prefill_ms:.3f} ms, decode step {step_ms:.3f} ms, decoded against prefilled {diff:.4f} (bound {BOUND})")
    sys.exit(0 if diff <= BOUND else 1)
