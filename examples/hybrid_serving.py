"""A small hybrid model served on the library: prompts, then one token at a time.

Three layers, each with a norm before it and a residual around it:

  KDA          short convolution over q, k and v, then the gated delta rule
  state space  short convolution over x, b and c, then the scan
  attention    keys and values in a paged cache, read by paged_decode

A batch of ragged prompts goes through packed; every layer then holds what it
needs to go on (a history, a state, a cache), and tokens follow one per
sequence. Weights are random and a token's input is a random vector, so the
check is one of the library against itself: the outputs of prompt + steps
equal those of one prompt that holds all the tokens, to bf16 rounding.

    python examples/hybrid_serving.py --prompts 300,37,1 --steps 16
    python examples/hybrid_serving.py --train          # gradients of the KDA layer too
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import prefill_kda_chunk_gb300 as K  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
WIDTH, TAPS, PAGE = 512, 4, 16


def norm(x):
    return torch.nn.functional.rms_norm(x.float(), (WIDTH,)).to(BF16)


class Layer:
    """Weights are drawn from a generator; `serve` keeps its state in self."""

    def __init__(self, gen):
        self.gen = gen

    def weight(self, rows, cols=WIDTH):
        w = torch.randn(rows, cols, generator=self.gen) / cols ** 0.5
        return w.to("cuda", BF16)

    def filters(self, channels):
        w = torch.randn(channels, TAPS, generator=self.gen) / TAPS ** 0.5
        return w.to("cuda")


class Kda(Layer):
    HEADS, DIM = 4, 128

    def __init__(self, gen):
        super().__init__(gen)
        inner = self.HEADS * self.DIM
        self.qkv, self.gate = self.weight(3 * inner), self.weight(inner)
        self.beta, self.out = self.weight(self.HEADS), self.weight(WIDTH, inner)
        self.conv = self.filters(3 * inner)

    def inputs(self, x, mixed):
        q, k, v = (t.reshape(-1, self.HEADS, self.DIM).contiguous()
                   for t in mixed.chunk(3, dim=-1))
        g = (x @ self.gate.T).float().reshape(-1, self.HEADS, self.DIM) + 3.0
        beta = torch.sigmoid((x @ self.beta.T).float())
        return q, k, v, g, beta

    def prompt(self, x, cu):
        mixed, self.history = K.short_conv(x @ self.qkv.T, self.conv, cu_seqlens=cu)
        o, self.state = K.chunk_prefill(*self.inputs(x, mixed), cu_seqlens=cu,
                                        normalize_qk=True, gate_logits=True)
        return o.reshape(-1, self.HEADS * self.DIM) @ self.out.T

    def step(self, x):
        mixed, self.history = K.short_conv_step(x @ self.qkv.T, self.conv, self.history,
                                                in_place=True)
        o, self.state = K.decode_step(*self.inputs(x, mixed), state=self.state, in_place=True,
                                      normalize_qk=True, gate_logits=True)
        return o.reshape(-1, self.HEADS * self.DIM) @ self.out.T


class StateSpace(Layer):
    HEADS, DIM, GROUPS, N = 8, 64, 2, 64

    def __init__(self, gen):
        super().__init__(gen)
        inner = self.HEADS * self.DIM
        self.sizes = [inner, self.GROUPS * self.N, self.GROUPS * self.N]
        self.xbc, self.dt = self.weight(sum(self.sizes)), self.weight(self.HEADS)
        self.out, self.conv = self.weight(WIDTH, inner), self.filters(sum(self.sizes))
        self.a = -torch.linspace(1.0, 8.0, self.HEADS, device="cuda")
        self.d = torch.ones(self.HEADS, device="cuda")
        self.dt_bias = torch.full((self.HEADS,), -3.0, device="cuda")

    def inputs(self, x, mixed):
        # slices of one array: the scan takes their strides as they are
        xs, b, c = mixed.split(self.sizes, dim=-1)
        return (xs.unflatten(-1, (self.HEADS, self.DIM)), (x @ self.dt.T).float(), self.a,
                b.unflatten(-1, (self.GROUPS, self.N)), c.unflatten(-1, (self.GROUPS, self.N)))

    def prompt(self, x, cu):
        mixed, self.history = K.short_conv(x @ self.xbc.T, self.conv, cu_seqlens=cu)
        y, self.state = K.ssm_prefill(*self.inputs(x, mixed), self.d, self.dt_bias,
                                      cu_seqlens=cu, dt_softplus=True)
        return y.reshape(-1, self.HEADS * self.DIM) @ self.out.T

    def step(self, x):
        mixed, self.history = K.short_conv_step(x @ self.xbc.T, self.conv, self.history,
                                                in_place=True)
        y, self.state = K.ssm_step(*self.inputs(x, mixed), state=self.state, d=self.d,
                                   dt_bias=self.dt_bias, dt_softplus=True, in_place=True)
        return y.reshape(-1, self.HEADS * self.DIM) @ self.out.T


class Attention(Layer):
    HEADS, KV_HEADS, DIM = 16, 2, 64

    def __init__(self, gen, longest, sequences):
        super().__init__(gen)
        self.q = self.weight(self.HEADS * self.DIM)
        self.kv = self.weight(2 * self.KV_HEADS * self.DIM)
        self.out = self.weight(WIDTH, self.HEADS * self.DIM)
        per = (longest + PAGE - 1) // PAGE
        # the pages of one cache, dealt out to the sequences in no order
        self.cache = torch.zeros(sequences * per, 2, PAGE, self.KV_HEADS, self.DIM,
                                 dtype=BF16, device="cuda")
        self.table = torch.randperm(sequences * per, generator=gen).to("cuda", torch.int32)
        self.table = self.table.view(sequences, per)

    def attend(self, x, seq, pos):
        """Token i is at position pos[i] of sequence seq[i]; its key and value join the
        cache, and it sees that sequence's tokens up to itself."""
        kv = (x @ self.kv.T).view(-1, 2, self.KV_HEADS, self.DIM)
        self.cache[self.table[seq, pos // PAGE].long(), :, pos % PAGE] = kv
        q = (x @ self.q.T).view(-1, self.HEADS, self.DIM)
        o, _ = K.paged_decode(q, self.cache[:, 0], self.cache[:, 1], self.table[seq],
                              (pos + 1).to(torch.int32))
        return o.reshape(-1, self.HEADS * self.DIM) @ self.out.T

    def prompt(self, x, cu):
        lens = (cu[1:] - cu[:-1]).long()
        seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), lens)
        pos = torch.arange(len(x), device="cuda") - cu[:-1].long()[seq]
        self.at = lens
        return self.attend(x, seq, pos)

    def step(self, x):
        o = self.attend(x, torch.arange(len(x), device="cuda"), self.at)
        self.at = self.at + 1
        return o


class Model:
    def __init__(self, seed, longest, sequences):
        gen = torch.Generator().manual_seed(seed)
        self.layers = [Kda(gen), StateSpace(gen), Attention(gen, longest, sequences)]

    def prompt(self, x, cu):
        for layer in self.layers:
            x = x + layer.prompt(norm(x), cu)
        return x

    def step(self, x):
        for layer in self.layers:
            x = x + layer.step(norm(x))
        return x


def serve(prompts, steps, seed=1):
    """The largest difference of prompt + steps from one prompt, over the largest value."""
    gen = torch.Generator().manual_seed(seed)
    tokens = [torch.randn(n + steps, WIDTH, generator=gen).to("cuda", BF16) for n in prompts]

    def cu(lens):
        return torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)

    model = Model(seed, max(prompts) + steps, len(prompts))
    got = [[row] for row in model.prompt(torch.cat([t[:n] for t, n in zip(tokens, prompts)]),
                                         cu(prompts)).split(prompts)]
    for i in range(steps):
        out = model.step(torch.stack([t[n + i] for t, n in zip(tokens, prompts)]))
        for rows, row in zip(got, out):
            rows.append(row[None])
    K.check_device_error()

    whole = Model(seed, max(prompts) + steps, len(prompts))
    lens = [n + steps for n in prompts]
    ref = whole.prompt(torch.cat(tokens), cu(lens))
    K.check_device_error()
    diff = (torch.cat([torch.cat(rows) for rows in got]).float() - ref.float()).abs().max()
    return float(diff / ref.float().abs().max())


def train(tokens=512, rounds=8, rate=0.5, seed=2):
    """Finds the filters of v in front of a KDA layer again from the layer's outputs, by
    the gradients of both; returns the loss before and after."""
    gen = torch.Generator().manual_seed(seed)
    layer, target = Kda(gen), None
    x = torch.randn(tokens, WIDTH, generator=gen).to("cuda", BF16)
    projected, losses = x @ layer.qkv.T, []
    for i in range(rounds + 1):
        mixed, _ = K.short_conv(projected, layer.conv)
        q, k, v, g, beta = layer.inputs(x, mixed)
        g = torch.nn.functional.logsigmoid(g)
        scale = Kda.DIM ** -0.5
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(BF16) for t in (q, k))
        o, _ = K.chunk_prefill(q, k, v, g, beta, scale=scale)
        if target is None:   # the filters to be found; start elsewhere
            target = o.float()
            layer.conv[2 * Kda.HEADS * Kda.DIM:] += 0.3 * layer.filters(Kda.HEADS * Kda.DIM)
            continue
        err = o.float() - target
        losses.append(float((err ** 2).mean() / (target ** 2).mean()))
        grads = K.chunk_prefill_backward(q, k, v, g, beta, err.to(BF16), scale=scale)
        # (those of q and k would go through the normalisation; they are at the target)
        d_mixed = torch.cat([torch.zeros_like(grads[0]), torch.zeros_like(grads[1]), grads[2]],
                            dim=-2).reshape(tokens, -1)
        _, d_conv = K.short_conv_backward(projected, layer.conv, d_mixed)[:2]
        layer.conv = layer.conv - rate * d_conv / d_conv.norm()
    K.check_device_error()
    return losses[0], losses[-1]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompts", default="300,37,1", help="tokens of each prompt")
    ap.add_argument("--steps", type=int, default=16, help="tokens after the prompts")
    ap.add_argument("--train", action="store_true", help="take gradient steps as well")
    a = ap.parse_args()
    worst = serve([int(n) for n in a.prompts.split(",")], a.steps)
    print(f"prompt + {a.steps} steps against one prompt: largest difference {worst:.2e} of the largest value")
    if a.train:
        print("filters in front of KDA, relative loss: %.3e -> %.3e" % train())


if __name__ == "__main__":
    main()
