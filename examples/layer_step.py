"""Training steps of an attention layer's query and key projection, replayable bit for bit.

    python examples/layer_step.py [--steps 5] [--seed 0]

The steps run the library's operators in the order a training program would: the projection (repro_gemm), the norm
of every query and key head with the position rotation (repro_rope_table, repro_qk_norm_rope), their gradients
(repro_qk_norm_rope_backward), the weight's gradient (repro_gemm), the clip of all gradients to a global norm
(GradList, repro_clip_grad_list) and AdamW with the state's hash (repro_adamw_hash).  The loss is half the squared
distance of the rotated heads from fixed targets.  The program trains twice from one seed and compares the hashes.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bitwise_reproducible_amd as br  # noqa: E402


class Layer:
    """Weights, gradients and optimizer state of the projection, each in one flat buffer with views of its parts."""

    def __init__(self, batch=2, seq=128, width=256, q_heads=8, k_heads=2, dim=64, seed=0):
        self.batch, self.seq, self.q_heads = batch, seq, q_heads
        heads = q_heads + k_heads
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(*shape, generator=gen, device="cuda") * std

        sizes = [width * heads * dim, dim, dim]
        n = sum(sizes)
        self.state = torch.zeros(3 * n, device="cuda")  # [w | m | v]
        self.grad = torch.zeros(n, device="cuda")
        weight, q_gain, k_gain = self.state[:n].split(sizes)
        self.weight, self.q_gain, self.k_gain = weight.view(width, heads * dim), q_gain, k_gain
        self.weight.copy_(normal(width, heads * dim, std=width ** -0.5))
        self.q_gain.fill_(1.0)
        self.k_gain.fill_(1.0)
        dweight, self.dq_gain, self.dk_gain = self.grad.split(sizes)
        self.dweight = dweight.view(width, heads * dim)
        self.clip = br.GradList([dweight, self.dq_gain, self.dk_gain])  # in place
        self.x = normal(batch * seq, width)
        self.projected = torch.empty(batch * seq, heads * dim, device="cuda")
        self.dprojected = torch.empty_like(self.projected)
        self.targets = normal(batch, seq, heads, dim)
        inv_freq = 5e5 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
        self.cos, self.sin = br.repro_rope_table(inv_freq, seq)
        self.shape = (batch, seq, heads, dim)
        self.digest = torch.empty(32, dtype=torch.uint8, device="cuda")
        self.workspace = br.hash_workspace(3 * n)
        self.norm = torch.empty(3, device="cuda")
        self.steps = 0

    def _sides(self, packed):
        """The query and the key heads of a packed (tokens, heads * dim) tensor, where they lie."""
        heads = packed.view(self.shape)
        return heads[:, :, :self.q_heads], heads[:, :, self.q_heads:]

    def step(self):
        """One step; the loss before it, as a device scalar."""
        br.repro_gemm(self.x, self.weight, out=self.projected)
        q, k = self._sides(self.projected)
        out = torch.empty(self.shape, device="cuda")
        q_out, k_out = self._sides(out)
        br.repro_qk_norm_rope(q, k, self.cos, self.sin, q_gain=self.q_gain, k_gain=self.k_gain, q_out=q_out,
                              k_out=k_out)
        away = out - self.targets  # the gradient of the loss
        dq, dk = self._sides(self.dprojected)
        dq_out, dk_out = self._sides(away)
        br.repro_qk_norm_rope_backward(q, k, dq_out, dk_out, self.cos, self.sin, q_gain=self.q_gain,
                                       k_gain=self.k_gain, dq=dq, dk=dk, dq_gain=self.dq_gain, dk_gain=self.dk_gain)
        br.repro_gemm(self.x, self.dprojected, trans_a=True, out=self.dweight)
        br.repro_clip_grad_list(self.clip, 1.0, out=self.norm)
        self.steps += 1
        br.repro_adamw_hash(self.state, self.grad, self.digest, self.workspace, lr=1e-2, beta1=0.9, beta2=0.95,
                            eps=1e-8, weight_decay=0.0, step=self.steps)
        return 0.5 * away.square().sum()


def train(steps, seed=0, tell=None, **sizes):
    """The state's hash and the loss of every step."""
    layer = Layer(seed=seed, **sizes)
    hashes, losses = [], []
    for i in range(steps):
        loss = layer.step()
        hashes.append(layer.digest.cpu().numpy().tobytes().hex())
        losses.append(loss.item())
        if tell:
            tell(f"step {i + 1}: loss {losses[-1]:.4f}  norm {layer.norm[0].item():.4f}  "
                 f"clipped by {layer.norm[2].item():.4f}  state {hashes[-1][:16]}...")
    return hashes, losses


def main():
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=5)
    parser.add_argument("--seed", type=int, default=0)
    args = parser.parse_args()
    first, _ = train(args.steps, args.seed, tell=print)
    again, _ = train(args.steps, args.seed)
    print("replayed bit for bit" if first == again else "THE REPLAY DIFFERS")
    return 0 if first == again else 1


if __name__ == "__main__":
    sys.exit(main())
