"""A small model over mel frames: trained on packed recordings, then run live.

Recordings become mel frames (MelSpectrogram), several of them packed into each
row of a batch. A causal transformer predicts every frame from the frames before
it: layer_norm before each block, attention with a learned bias by distance
and the recordings kept apart by document ids. The trained model then takes a
recording one frame at a time against a cache of keys and values, which gives
the same predictions.

    python examples/frame_encoder.py [--steps 20] [--dtype bf16]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mel_spectrogram_gb300 import FM_OK, MelSpectrogram, attention, layer_norm, ops  # noqa: E402


class Norm(nn.Module):
    def __init__(self, width):
        super().__init__()
        self.weight = nn.Parameter(torch.ones(width))
        self.bias = nn.Parameter(torch.zeros(width))

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias)


class Block(nn.Module):
    def __init__(self, width, heads, kv_heads, buckets):
        super().__init__()
        self.heads, self.kv_heads, self.dim = heads, kv_heads, width // heads
        self.norm1, self.norm2 = Norm(width), Norm(width)
        self.qkv = nn.Linear(width, (heads + 2 * kv_heads) * self.dim)
        self.out = nn.Linear(width, width)
        self.mlp = nn.Sequential(nn.Linear(width, 4 * width), nn.GELU(), nn.Linear(4 * width, width))
        self.table = nn.Parameter(torch.zeros(buckets, heads))

    def split(self, x):
        qkv = self.qkv(self.norm1(x)).unflatten(-1, (-1, self.dim))
        return qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=2)

    def finish(self, x, a):
        x = x + self.out(a.flatten(2))
        return x + self.mlp(self.norm2(x))

    def forward(self, x, documents):
        q, k, v = self.split(x)
        a = attention(q, k, v, causal=True, q_start=0, q_docs=documents, k_docs=documents, table=self.table,
                      max_distance=MAX_DISTANCE, bidirectional=False)
        return self.finish(x, a)

    def step(self, x, keys, values, lens):
        """New frames x (batch, n, width) of streams whose caches hold lens - n frames so far."""
        q, k, v = self.split(x)
        place = (lens - x.shape[1])[:, None] + torch.arange(x.shape[1], device=x.device, dtype=torch.int32)
        rows = torch.arange(x.shape[0], device=x.device)[:, None]
        keys[rows, place], values[rows, place] = k, v
        a = attention(q, keys, values, causal=True, k_lens=lens, table=self.table, max_distance=MAX_DISTANCE,
                      bidirectional=False)
        return self.finish(x, a)


MAX_DISTANCE = 400  # frames: 4 s at hop 160


class FrameModel(nn.Module):
    def __init__(self, n_mels=80, width=256, heads=4, kv_heads=2, blocks=2, buckets=32):
        super().__init__()
        self.embed = nn.Linear(n_mels, width)
        self.blocks = nn.ModuleList(Block(width, heads, kv_heads, buckets) for _ in range(blocks))
        self.norm = Norm(width)
        self.head = nn.Linear(width, n_mels)

    def forward(self, frames, documents):
        x = self.embed(frames)
        for b in self.blocks:
            x = b(x, documents)
        return self.head(self.norm(x))

    def cache(self, batch, frames):
        like = self.embed.weight
        return [torch.zeros(2, batch, frames, b.kv_heads, b.dim, dtype=like.dtype, device=like.device)
                for b in self.blocks]

    def step(self, frames, cache, lens):
        x = self.embed(frames)
        for b, (keys, values) in zip(self.blocks, cache):
            x = b.step(x, keys, values, lens)
        return self.head(self.norm(x))


def recordings(n, seconds, seed):
    """Chirps with noise, n of them, of uneven length."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for k in range(n):
        t = torch.arange(int(16000 * seconds * (0.5 + 0.5 * (k + 1) / n)), device="cuda") / 16000
        f = 200 + 1500 * torch.rand(2, device="cuda", generator=g)
        x = torch.sin(6.2832 * (f[0] * t + f[1] * t * t / (2 * seconds)))
        out.append(x + 0.05 * torch.randn(x.shape, device="cuda", generator=g))
    return out


def pack(frames, rows):
    """Recordings' frames laid end to end in `rows` rows: (frames, document ids)."""
    per = [frames[r::rows] for r in range(rows)]
    longest = max(sum(len(f) for f in row) for row in per)
    batch = torch.zeros(rows, longest, frames[0].shape[1], dtype=frames[0].dtype, device="cuda")
    ids = torch.full((rows, longest), -1, dtype=torch.int32, device="cuda")
    for r, row in enumerate(per):
        at = 0
        for n, f in enumerate(row):
            batch[r, at:at + len(f)], ids[r, at:at + len(f)] = f, n
            at += len(f)
    return batch, ids


def run(steps=20, dtype=torch.bfloat16, seconds=2.0, seed=0):
    """Train, then stream; returns the losses and how far the streamed
    predictions are from the packed pass (relative)."""
    torch.manual_seed(seed)
    mel = MelSpectrogram(sample_rate=16000, n_fft=400, hop_length=160, n_mels=80)
    with torch.no_grad():
        frames = [torch.log(mel(x) + 1e-3).t().to(dtype) for x in recordings(6, seconds, seed)]
    batch, ids = pack(frames, rows=2)
    model = FrameModel().to("cuda", dtype)
    optimiser = torch.optim.AdamW(model.parameters(), lr=1e-3)
    known = ((ids[:, 1:] == ids[:, :-1]) & (ids[:, 1:] >= 0))[..., None]
    losses = []
    for _ in range(steps):
        optimiser.zero_grad(set_to_none=True)
        error = (model(batch, ids)[:, :-1] - batch[:, 1:]).float()
        loss = torch.where(known, error, 0.0).square().sum() / (known.sum() * batch.shape[2])
        loss.backward()
        optimiser.step()
        losses.append(float(loss.detach()))
    with torch.no_grad():
        first = frames[0][None]
        whole = model(first, torch.zeros(1, first.shape[1], dtype=torch.int32, device="cuda"))
        cache, got = model.cache(1, first.shape[1]), []
        for n in range(first.shape[1]):
            lens = torch.full((1,), n + 1, dtype=torch.int32, device="cuda")
            got.append(model.step(first[:, n:n + 1], cache, lens))
        far = float((torch.cat(got, 1) - whole).float().norm() / whole.float().norm())
    if ops.poll_error() != FM_OK:
        raise RuntimeError("a wait in a kernel gave up: the results are not valid")
    return losses, far


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--dtype", choices=["f32", "f16", "bf16"], default="bf16")
    a = p.parse_args()
    losses, far = run(a.steps, {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[a.dtype])
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps; "
          f"streamed against packed predictions: relative {far:.2g}")
