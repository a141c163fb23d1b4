"""A small language model with a sparse expert layer, trained and sampled from
with this package's operators:

    tokens -> embedding -> router -> tokens sorted by expert -> experts -> back, weighted -> logits -> top-k

    python examples/sparse_layer.py [--steps 60] [--dtype bfloat16]

The data is synthetic (each token is followed by a fixed other one most of the
time), so the loss has a known floor. In 16 bits the experts' products run in
libsegtopk.so too, from the experts' offsets on the device; in 32 bits they are
torch matrix products, expert by expert. The logits are torch's. The five
autograd functions below are all that is needed to use the operators in a
model that torch differentiates.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import segmented_radix_top_gb300 as st  # noqa: E402


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, tokens, scale):
        ctx.save_for_backward(tokens)
        ctx.rows, ctx.scale, ctx.dtype = table.shape[0], scale, table.dtype
        return st.embedding(table, tokens, scale=scale)

    @staticmethod
    def backward(ctx, grad):
        tokens, = ctx.saved_tensors
        return st.embedding_backward(grad, tokens, ctx.rows, scale=ctx.scale, dtype=ctx.dtype), None, None


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k):
        ids, weights = st.route(logits, k)
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    def backward(ctx, _, grad):
        logits, ids = ctx.saved_tensors
        return st.route_backward(grad, logits, ids), None


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, groups):
        ctx.groups = groups
        return st.dispatch(x, groups)

    @staticmethod
    def backward(ctx, grad):
        return st.dispatch_backward(grad, ctx.groups), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, groups):
        ctx.save_for_backward(rows, weights)
        ctx.groups = groups
        return st.combine(rows, groups, weights)

    @staticmethod
    def backward(ctx, grad):
        rows, weights = ctx.saved_tensors
        return *st.combine_backward(grad, rows, ctx.groups, weights), None


class Product(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, groups):
        ctx.save_for_backward(rows, weights)
        ctx.groups = groups
        return st.expert_matmul(rows, weights, groups)

    @staticmethod
    def backward(ctx, grad):
        return *st.expert_matmul_backward(grad, *ctx.saved_tensors, ctx.groups), None


class SparseModel(torch.nn.Module):
    def __init__(self, vocab, width, hidden, experts, k, device="cuda", seed=0, dtype=torch.float32):
        super().__init__()
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, scale):
            return torch.nn.Parameter((scale * torch.randn(*shape, generator=g)).to(device, dtype))

        self.k = k
        self.table = weight(vocab, width, scale=width ** -0.5)
        self.router = weight(width, experts, scale=width ** -0.5)
        self.up = weight(experts, width, hidden, scale=width ** -0.5)
        self.down = weight(experts, hidden, width, scale=hidden ** -0.5)
        self.head = weight(width, vocab, scale=width ** -0.5)

    def experts(self, rows, groups):
        """Each expert's two products on its rows; rows of no expert stay zero."""
        if rows.dtype != torch.float32:
            hidden = Product.apply(rows, self.up.transpose(1, 2), groups)
            return Product.apply(torch.nn.functional.gelu(hidden), self.down.transpose(1, 2), groups)
        bounds = groups.offsets.tolist()
        done = [torch.nn.functional.gelu(rows[a:b] @ self.up[e]) @ self.down[e]
                for e, (a, b) in enumerate(zip(bounds, bounds[1:]))]
        return torch.cat(done + [rows[bounds[-1]:]])

    def forward(self, tokens):
        x = Embedding.apply(self.table, tokens, self.table.shape[1] ** 0.5)
        ids, weights = Route.apply(x @ self.router, self.k)
        groups = st.group_by_expert(ids, self.router.shape[1])
        rows = self.experts(Dispatch.apply(x, groups), groups)
        return (x + Combine.apply(rows, weights, groups)) @ self.head


def sample(model, tokens, k, generator):
    """One more token for each of `tokens`: drawn from the k most likely (the segmented top-k of the rows of logits)."""
    logits = model(tokens)
    rows, vocab = logits.shape
    offsets = torch.arange(0, (rows + 1) * vocab, vocab, device=logits.device)
    ids = torch.arange(vocab, dtype=torch.int32, device=logits.device).repeat(rows)
    best, which = st.batched_topk(logits.reshape(-1), offsets, k, values=ids, max_segment_len=vocab)
    p = torch.softmax(best.reshape(rows, k).float(), 1)
    return which.reshape(rows, k).gather(1, torch.multinomial(p, 1, generator=generator)).squeeze(1)


def text(n, vocab, generator, device="cuda"):
    """Pairs (token, next): next is 7 token + 3 modulo vocab nine times in ten, else any."""
    tokens = torch.randint(0, vocab, (n,), generator=generator, device=device)
    other = torch.randint(0, vocab, (n,), generator=generator, device=device)
    rule = torch.rand(n, generator=generator, device=device) < 0.9
    return tokens, torch.where(rule, (7 * tokens + 3) % vocab, other)


def train(steps=60, vocab=512, width=128, hidden=256, experts=16, k=2, batch=4096, rate=2e-3, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(1)
    model = SparseModel(vocab, width, hidden, experts, k, dtype=dtype)
    optimizer = torch.optim.Adam(model.parameters(), lr=rate)
    losses = []
    for _ in range(steps):
        tokens, following = text(batch, vocab, g)
        loss = torch.nn.functional.cross_entropy(model(tokens).float(), following)
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(float(loss.detach()))
    tokens = torch.arange(vocab, device="cuda")
    with torch.no_grad():
        right = (sample(model, tokens, 5, g) == (7 * tokens + 3) % vocab).float().mean()
    return losses, float(right)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    # float16 would want a loss scale and an optimizer in 32 bits: Adam's 1e-8 is 0 there
    ap.add_argument("--dtype", choices=["float32", "bfloat16"], default="float32")
    args = ap.parse_args()
    losses, right = train(args.steps, dtype=getattr(torch, args.dtype))
    print("loss %.3f -> %.3f; %.0f %% of the sampled tokens follow the rule" % (losses[0], losses[-1], 100 * right))


if __name__ == "__main__":
    main()
