"""A small language model trained on the DBuffer step's own formats, on one GPU.

    python examples/fp8_lm.py [--steps 60] [--layers 2] [--width 512] [--vocab 1000]

Every weight is read as the optimizer step leaves it: E4M3 codes with one scale per
128 x 128 tile, at its place in the FP8 staging buffer (the AllGather's result, here of
one device).  The forward pass is lookup, residual norm with FP8 rows, and FP8
projections, and a loss over the head that keeps no logits (cross entropy, or the divergence
from a teacher's top logits); the backward pass the operators' gradients, bf16, which the pack
and the 8-bit Adam step turn into the next codes.  torch does the elementwise rest: the
squared ReLU.

The task: the next token is a fixed permutation of the current one, so the loss falls
from log(vocab) towards zero.
"""

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import block_quant_gb300 as bq  # noqa: E402

EPS = 1e-5


class Model:
    """Embedding, `layers` of (norm, up, squared ReLU, down) with residuals, a last norm
    and a head, for batches of `tokens` tokens."""

    def __init__(self, vocab, width, hidden, layers, tokens, device, seed=0):
        self.vocab, self.width, self.hidden, self.layers, self.n = vocab, width, hidden, layers, tokens
        self.dev = device
        shapes = {"embed": (vocab, width)}
        for i in range(layers):
            shapes[f"norm{i}"] = (1, width)
            shapes[f"up{i}"] = (hidden, width)
            shapes[f"down{i}"] = (width, hidden)
        shapes["norm"] = (1, width)
        shapes["head"] = (vocab, width)
        self.shapes, self.names = shapes, list(shapes)

        # one device's DBuffer: FP8 tiles for the matrices, none for the norms
        descs = []
        for r, c in shapes.values():
            two = r > 1
            descs.append((r, c, math.lcm(128 * c, 256) if two else 256, bq.ADAM_FLAT256, int(two)))
        self.layout = bq.plan(descs, 1)
        table = self.layout.export()
        n, ni, nm, nf, size = int(table[4]), int(table[5]), int(table[6]), int(table[7]), int(table[3])
        rows = table[8 + 7 * n: 8 + 7 * n + 7 * ni].reshape(ni, 7)  # dev, tensor, t_off, len, local_off, mslot, fslot
        self.place = {self.names[int(r[1])]: (int(r[4]), int(r[6])) for r in rows}

        new = lambda k, dt: torch.zeros(k, dtype=dt, device=device)  # noqa: E731
        self.tables = torch.empty(self.layout.upload_bytes(0, 1), dtype=torch.uint8, device=device)
        self.shard = self.layout.upload(0, 1, self.tables)
        self.master, self.dbuf = new(size, torch.float32), new(size, torch.bfloat16)
        self.m, self.v = new(size, torch.int8), new(size, torch.uint8)
        self.m_scale, self.v_scale = new(nm, torch.float32), new(nm, torch.float32)
        self.codes, self.scales = new(size, torch.uint8), new(max(nf, 1), torch.float32)
        gen = torch.Generator(device=device).manual_seed(seed)
        for name, (r, c) in shapes.items():
            at = self.place[name][0]
            w = self.master[at:at + r * c]
            if r == 1:
                w.fill_(1.0)
            else:
                w.copy_(torch.randn(r * c, generator=gen, device=device) * (1.0 if name == "embed" else c ** -0.5))
        bq.quant_fp8(self.shard, self.master, self.codes, self.scales)

        # gradients, one bf16 tensor a parameter, and their addresses for the pack
        self.grads = {k: new(r * c, torch.bfloat16).view(r, c) for k, (r, c) in shapes.items()}
        self.grad_ptrs = torch.tensor([g.data_ptr() for g in self.grads.values()], dtype=torch.int64, device=device)
        need = max(bq.linear_fp8_workspace(tokens, r, c) for r, c in shapes.values() if r > 1)
        self.ws = new(need, torch.uint8)
        self.ws_embed = new(bq.embed_grad_workspace(tokens, vocab, width), torch.uint8)
        self.ws_norm = new(bq.rmsnorm_grad_workspace(tokens, width), torch.uint8)
        self.ws_loss = new(bq.loss_fp8_workspace(tokens, vocab, width), torch.uint8)
        self.ws_loss_grad = new(bq.loss_fp8_grad_workspace(tokens, vocab, width), torch.uint8)
        self.t = 0

    # ------------------------------------------------------------------ parameters as gathered

    def weight(self, name):
        """(codes [rows, cols], tile scales) of a matrix in the staging buffer."""
        (r, c), (at, slot) = self.shapes[name], self.place[name]
        return self.codes[at:at + r * c].view(r, c), self.scales[slot:slot + -(-r // 128) * -(-c // 128)]

    def vector(self, name):
        at = self.place[name][0]
        return self.master[at:at + self.shapes[name][1]].bfloat16()

    # ------------------------------------------------------------------ pieces

    def _rows(self, c, dtype=torch.bfloat16):
        return torch.empty(self.n, c, dtype=dtype, device=self.dev)

    def _fp8_rows(self, c):
        return self._rows(c, torch.uint8), torch.empty(-(-c // 128), self.n, device=self.dev)

    def _norm(self, name, x, residual):
        h = self._rows(self.width) if residual is not None else x
        w, rstd = self.vector(name), torch.empty(self.n, device=self.dev)
        codes, scale = self._fp8_rows(self.width)
        bq.rmsnorm(x, w, EPS, residual=residual, h=h if residual is not None else None, codes=codes, code_scale=scale,
                   rstd=rstd)
        return h, (name, h, w, rstd), (codes, scale)

    def _linear(self, name, rows):
        out = self._rows(self.shapes[name][0])
        bq.linear_fp8(*rows, *self.weight(name), out, self.ws)
        return out

    def _linear_grad(self, name, dy, rows):
        dx = self._rows(self.shapes[name][1])
        bq.linear_fp8_dw(dy, *rows, self.grads[name], self.ws)
        bq.linear_fp8_dx(dy, *self.weight(name), dx, self.ws)
        return dx

    def _norm_grad(self, saved, dy, dh):
        name, h, w, rstd = saved
        dx = self._rows(self.width)
        bq.rmsnorm_grad(dy, h, w, rstd, dx, self.grads[name][0], self.ws_norm, dh=dh)
        return dx

    # ------------------------------------------------------------------ one step

    def encode(self, ids):
        """The last norm's FP8 rows, and what the backward pass needs."""
        x, h, tape = self._rows(self.width), None, []
        codes, scales = self.weight("embed")
        bq.embed(codes, ids, x, table_scale=scales)
        for i in range(self.layers):
            h, norm, rows = self._norm(f"norm{i}", x, h)
            u = self._linear(f"up{i}", rows)
            a = torch.relu(u).square()
            inner = self._fp8_rows(self.hidden)
            bq.quant_rows_fp8(a, *inner)
            x = self._linear(f"down{i}", inner)
            tape.append((norm, rows, u, inner))
        _, norm, rows = self._norm("norm", x, h)
        return rows, (tape, norm, rows)

    def forward(self, ids):
        rows, saved = self.encode(ids)
        return self._linear("head", rows), saved

    def backward(self, ids, dlogits, saved):
        """Fills self.grads from the gradient of the logits."""
        self.backward_rows(ids, self._linear_grad("head", dlogits, saved[2]), saved)

    def backward_rows(self, ids, drows, saved):
        """Fills self.grads but for the head's from the gradient of the last norm's output."""
        tape, norm, _ = saved
        dh = self._norm_grad(norm, drows, None)
        for i in reversed(range(self.layers)):
            norm, rows, u, inner = tape[i]
            da = self._linear_grad(f"down{i}", dh, inner)
            du = da * 2 * torch.relu(u)
            dh = self._norm_grad(norm, self._linear_grad(f"up{i}", du, rows), dh)
        bq.embed_grad(dh, ids, self.grads["embed"], self.ws_embed)

    def _vector(self):
        return torch.empty(self.n, device=self.dev)

    def cross_entropy(self, rows, targets, dloss):
        """Each token's loss and the gradient of rows; fills the head's."""
        head, loss, lse, dx = (*rows, *self.weight("head")), self._vector(), self._vector(), self._rows(self.width)
        bq.cross_entropy_fp8(*head, targets, loss, lse, self.ws_loss)
        bq.cross_entropy_fp8_grad(*head, targets, loss, lse, dloss, dx, self.grads["head"], self.ws_loss_grad)
        return loss, dx

    def distill(self, rows, ids, teacher, dloss, temperature=1.0):
        """The same against a teacher's top logits: ids and teacher [tokens, k]."""
        head, loss, lse, dx = (*rows, *self.weight("head")), self._vector(), self._vector(), self._rows(self.width)
        logp = torch.empty(ids.shape, device=self.dev)
        bq.distill_fp8(*head, ids, teacher, loss, lse, logp, self.ws_loss, scale=1 / temperature)
        bq.distill_fp8_grad(*head, ids, teacher, lse, logp, dloss, dx, self.grads["head"], self.ws_loss_grad,
                            scale=1 / temperature)
        return loss, dx

    def step(self, ids, targets, lr, eps, teacher=None):
        """One step on targets, or, with the teacher's logits [tokens, k] of them, on targets [tokens, k]."""
        rows, saved = self.encode(ids)
        dloss = torch.full((self.n,), 1 / self.n, device=self.dev)
        if teacher is None:
            loss, dx = self.cross_entropy(rows, targets, dloss)
        else:
            loss, dx = self.distill(rows, targets, teacher, dloss)
        self.backward_rows(ids, dx, saved)
        self.t += 1
        bq.pack(self.shard, self.grad_ptrs, self.dbuf, 1.0)
        hp = bq.adam_hparams(lr, 0.9, 0.95, eps, self.t)
        bq.step_adam8(self.shard, self.dbuf, self.master, self.m, self.v, self.m_scale, self.v_scale, hp, self.codes,
                      self.scales)
        return loss.mean()

    def check(self):
        """Raises if a device wait of the steps so far gave up."""
        for ws in (self.ws, self.ws_loss, self.ws_loss_grad):
            bq.linear_check(ws)
        bq.shard_check(self.shard)


def train(steps, vocab=1000, width=512, hidden=1024, layers=2, tokens=2048, lr=2e-3, eps=1e-4, seed=0, tell=None):
    """Losses of `steps` steps on the permutation task.  (The second moment is linear in
    its block, so its small values are codes of 0 and eps is what bounds their step.)"""
    dev = torch.device("cuda")
    model = Model(vocab, width, hidden, layers, tokens, dev, seed)
    rng = np.random.default_rng(seed)
    after = torch.as_tensor(rng.permutation(vocab)).to(dev)
    losses = []
    for i in range(steps):
        ids = torch.as_tensor(rng.integers(0, vocab, tokens)).to(dev)
        losses.append(model.step(ids, after[ids], lr, eps))
        if tell and (i % 10 == 0 or i + 1 == steps):
            tell(i, float(losses[-1]))
    model.check()
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=1000)
    a = ap.parse_args()
    train(a.steps, vocab=a.vocab, width=a.width, hidden=2 * a.width, layers=a.layers,
          tell=lambda i, loss: print(f"step {i:4d}  loss {loss:.4f}"))
