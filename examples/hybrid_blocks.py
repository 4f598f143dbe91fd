"""A small language model of two kinds of recurrent blocks, trained, prompted and decoded token by token with this library.

Each block adds its predecessor's output to the residual stream and normalises it (``add_rms_norm``), mixes tokens with a
short convolution and a recurrence, and ends in an output projection:

* ``DeltaBlock``: convolution -> gated delta rule -> gated norm per head (``gated_rms_norm``);
* ``ScanBlock``: convolution -> selective scan, whose own gate and skip close it.

A prompt leaves each block's states (``causal_conv1d_state`` and the recurrence's final state); decoding carries them on with
``causal_conv1d_step``, ``gdn_step`` and ``selective_scan_step``. Run on a GB300: ``python examples/hybrid_blocks.py``.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_05_gb300 as lib  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
TAPS = 4


def parameter(*shape, std, dtype=BF16, mean=0.0):
    return (mean + std * torch.randn(*shape, device="cuda")).to(dtype).requires_grad_()


class DeltaBlock:
    def __init__(self, heads, qk_heads, scale):
        self.H, self.Hk, self.scale = heads, qk_heads, scale
        width, self.C = heads * 128, (heads + 2 * qk_heads) * 128
        self.p = {
            "norm": parameter(width, std=0, mean=1, dtype=F32), "w_in": parameter(width, self.C + width + 2 * heads, std=width ** -0.5),
            "conv": parameter(self.C, TAPS, std=0.3, dtype=F32), "out_norm": parameter(128, std=0, mean=1, dtype=F32),
            "w_out": parameter(width, width, std=width ** -0.5),
        }

    def split(self, y):
        mixed, gate, g, beta = (y @ self.p["w_in"]).split([self.C, self.H * 128, self.H, self.H], -1)
        return mixed.contiguous(), gate, -torch.nn.functional.softplus(g.float()), torch.sigmoid(beta)

    def heads(self, mixed):
        q, k, v = mixed.split([self.Hk * 128, self.Hk * 128, self.H * 128], -1)
        shape = mixed.shape[:-1]
        return q.reshape(*shape, self.Hk, 128), k.reshape(*shape, self.Hk, 128), v.reshape(*shape, self.H, 128)

    def close(self, o, gate):
        o = lib.gated_rms_norm(o.contiguous(), gate.reshape(o.shape).contiguous(), self.p["out_norm"])
        return o.flatten(-2) @ self.p["w_out"]

    def prompt(self, x, stream, keep):
        y, stream = lib.add_rms_norm(x, stream, self.p["norm"], residual_scale=self.scale)
        mixed, gate, g, beta = self.split(y)
        q, k, v = (t.contiguous() for t in self.heads(lib.causal_conv1d(mixed, self.p["conv"])))
        o, S = lib.chunk_gated_delta_rule(q, k, v, g.contiguous(), beta.contiguous(), output_final_state=keep)
        return self.close(o, gate), stream, (lib.causal_conv1d_state(mixed, self.p["conv"]), S) if keep else None

    def step(self, x, stream, cache):
        conv, S = cache
        y, stream = lib.add_rms_norm_fwd(x, stream, self.p["norm"], residual_scale=self.scale)
        mixed, gate, g, beta = self.split(y)
        q, k, v = self.heads(lib.causal_conv1d_step(conv, mixed, self.p["conv"]))
        return self.close(lib.gdn_step(S, q, k, v, g.contiguous(), beta.contiguous()), gate), stream


class ScanBlock:
    def __init__(self, width, channels, states, rank, scale):
        self.E, self.N, self.R, self.scale = channels, states, rank, scale
        step = torch.exp(torch.rand(channels, device="cuda") * 4.6 - 6.9)      # 0.001 .. 0.1
        self.p = {
            "norm": parameter(width, std=0, mean=1, dtype=F32), "w_in": parameter(width, 2 * channels, std=width ** -0.5),
            "conv": parameter(channels, TAPS, std=0.3, dtype=F32), "w_x": parameter(channels, rank + 2 * states, std=channels ** -0.5),
            "w_dt": parameter(rank, channels, std=rank ** -0.5), "dt_bias": (step + torch.log(-torch.expm1(-step))).requires_grad_(),
            "A_log": torch.log(torch.arange(1, states + 1, device="cuda", dtype=F32)).repeat(channels, 1).requires_grad_(),
            "D": parameter(channels, std=0, mean=1, dtype=F32), "w_out": parameter(channels, width, std=channels ** -0.5),
        }

    def split(self, u):
        low, B, C = (u @ self.p["w_x"]).split([self.R, self.N, self.N], -1)     # B and C stay strided slices
        return low @ self.p["w_dt"], -torch.exp(self.p["A_log"]), B.unsqueeze(-2), C.unsqueeze(-2)

    def prompt(self, x, stream, keep):
        y, stream = lib.add_rms_norm(x, stream, self.p["norm"], residual_scale=self.scale)
        v, z = (y @ self.p["w_in"]).split([self.E, self.E], -1)
        v = v.contiguous()
        u = lib.causal_conv1d(v, self.p["conv"])
        delta, A, B, C = self.split(u)
        o, h = lib.selective_scan(u, delta, A, B, C, D=self.p["D"], z=z, delta_bias=self.p["dt_bias"], output_final_state=keep)
        return o @ self.p["w_out"], stream, (lib.causal_conv1d_state(v, self.p["conv"]), h) if keep else None

    def step(self, x, stream, cache):
        conv, h = cache
        y, stream = lib.add_rms_norm_fwd(x, stream, self.p["norm"], residual_scale=self.scale)
        v, z = (y @ self.p["w_in"]).split([self.E, self.E], -1)
        u = lib.causal_conv1d_step(conv, v, self.p["conv"])
        delta, A, B, C = self.split(u)
        return lib.selective_scan_step(h, u, delta, A, B, C, D=self.p["D"], z=z, delta_bias=self.p["dt_bias"]) @ self.p["w_out"], stream


class Model:
    def __init__(self, vocab=512, heads=2, qk_heads=1, channels=384, states=16, rank=16, pairs=2):
        width = heads * 128
        scale = (2 * pairs) ** -0.5
        self.embed = parameter(vocab, width, std=1.0)
        self.norm = parameter(width, std=0, mean=1, dtype=F32)
        self.blocks = [b for _ in range(pairs) for b in (DeltaBlock(heads, qk_heads, scale), ScanBlock(width, channels, states, rank, scale))]

    def parameters(self):
        return [self.embed, self.norm, *(t for b in self.blocks for t in b.p.values())]

    def logits(self, x, stream):
        y, _ = lib.add_rms_norm(x, stream, self.norm)
        return y @ self.embed.t() * self.embed.shape[1] ** -0.5

    def prompt(self, tokens, keep=False):
        """Logits of every token of ``tokens [B,T]``, and the blocks' states after it."""
        x = self.embed[tokens]
        stream, x, caches = x.float(), torch.zeros_like(x), []
        for b in self.blocks:
            x, stream, cache = b.prompt(x, stream, keep)
            caches.append(cache)
        return self.logits(x, stream), caches

    def step(self, tokens, caches):
        """Logits of one more token per sequence ``[B]``; the states are carried on in place."""
        x = self.embed[tokens]
        stream, x = x.float(), torch.zeros_like(x)
        for b, cache in zip(self.blocks, caches):
            x, stream = b.step(x, stream, cache)
        return self.logits(x, stream)


def train(model, tokens, steps, lr=3e-3):
    """Next-token training on ``tokens [B,T]``; the losses."""
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0)
    losses = []
    for _ in range(steps):
        logits, _ = model.prompt(tokens[:, :-1].contiguous())
        loss = torch.nn.functional.cross_entropy(logits.float().flatten(0, 1), tokens[:, 1:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


@torch.no_grad()
def decode(model, tokens, cut):
    """Logits of ``tokens [B,T]`` from a prompt of ``cut`` tokens and single-token steps for the rest."""
    logits, caches = model.prompt(tokens[:, :cut].contiguous(), keep=True)
    return torch.cat([logits, *(model.step(tokens[:, t], caches)[:, None] for t in range(cut, tokens.shape[1]))], 1)


def main():
    torch.manual_seed(0)
    model = Model()
    tokens = torch.randint(0, 512, (4, 257), device="cuda")
    losses = train(model, tokens, 30)
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps")
    with torch.no_grad():
        whole, _ = model.prompt(tokens)
        steps = decode(model, tokens, 200)
        off = (steps - whole).double().norm() / whole.double().norm()
        print(f"prompt of 200 tokens and 57 single steps against one prompt of 257: logits off by {off:.1e}, "
              f"same choice for {(steps.argmax(-1) == whole.argmax(-1)).float().mean():.1%} of the tokens")
        _, caches = model.prompt(tokens, keep=True)
        nxt = tokens[:, -1]
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(100):
            nxt = model.step(nxt, caches).argmax(-1)
        torch.cuda.synchronize()
        print(f"decoding: {(time.perf_counter() - t0) * 10:.2f} ms a token of {len(tokens)} sequences")


if __name__ == "__main__":
    main()
