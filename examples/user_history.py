"""Users' event histories beside pooled embeddings, with the entry points of
``dlrm_history.h`` and ``dlrm_sparse.h`` together.

    python examples/user_history.py

Serving: each user's past events lie in a paged key/value cache.  New events
are appended (their keys normed and rotated on the way) and attend over what
came before them; then candidate items attend over the whole history, and what
each gathers enters the pairwise interaction beside its user's pooled bag.
Training: the head norms' weights are fitted through the gradient call.
"""
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_dense_interaction_gb300 as sdi


class NormRope(torch.autograd.Function):
    """Head norm and rotation of queries and keys ``[n][heads][d]``, with gradients."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, eps, rope, positions):
        q_out, k_out = torch.empty_like(q), torch.empty_like(k)
        sdi.dlrm_qk_norm_rope_fwd(q, k, q_weight, k_weight, eps, rope, positions, q_out, k_out)
        ctx.save_for_backward(q, k, q_weight, k_weight, rope, positions)
        ctx.eps = eps
        return q_out, k_out

    @staticmethod
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, rope, positions = ctx.saved_tensors
        dq, dk = torch.empty_like(q), torch.empty_like(k)
        dq_weight, dk_weight = torch.empty_like(q_weight), torch.empty_like(k_weight)
        size = sdi.dlrm_qk_norm_rope_bwd_workspace_size(q.shape[0], q.shape[1], k.shape[1], q.shape[2])
        sdi.dlrm_qk_norm_rope_bwd(dq_out.contiguous(), dk_out.contiguous(), q, k, q_weight, k_weight, ctx.eps, rope,
                                  positions, dq, dk, dq_weight, dk_weight,
                                  torch.empty(size, dtype=torch.uint8, device=q.device))
        return dq, dk, dq_weight, dk_weight, None, None, None


class HistoryModel:
    """Random weights: an item table, projections to heads, norms, rotation."""

    def __init__(self, items=1000, width=64, q_heads=4, kv_heads=2, d=64, length=4096, dtype=torch.bfloat16, seed=0,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=g)
        self.q_heads, self.kv_heads, self.d, self.dtype, self.eps, self.device = q_heads, kv_heads, d, dtype, 1e-6, device
        self.table = rand(items, width).to(device)
        self.qkv = (rand(width, (q_heads + 2 * kv_heads) * d) / width ** 0.5).to(device)
        self.back = (rand(q_heads * d, width) / (q_heads * d) ** 0.5).to(device)
        self.q_weight, self.k_weight = ((1 + 0.2 * rand(d)).to(device) for _ in range(2))
        angles = torch.arange(length)[:, None] * 10000.0 ** (-torch.arange(0, d, 2) / d)
        self.rope = torch.cat([angles.cos(), angles.sin()], 1).to(device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)

    def heads(self, items):
        """Queries, keys and values of items: views of one projection."""
        offsets = torch.arange(items.numel() + 1, device=self.device)
        rows = torch.empty((items.numel(), 1, self.table.shape[1]), device=self.device)
        sdi.dlrm_emb_bag_fwd([self.table], offsets, items, items.numel(), rows, err_flag=self.err)
        x = (rows[:, 0] @ self.qkv).to(self.dtype).view(items.numel(), -1, self.d)
        return x.split([self.q_heads, self.kv_heads, self.kv_heads], 1)


class Histories:
    """The paged cache of a set of users, and who has which page."""

    def __init__(self, model, users, pages=256, page_size=16, pages_of_user=64):
        m = self.model = model
        shape = (pages, m.kv_heads, page_size, m.d)
        self.k, self.v = (torch.zeros(shape, dtype=m.dtype, device=m.device).transpose(1, 2) for _ in range(2))
        self.free, self.page_size = list(range(pages)), page_size
        self.lengths = [0] * users
        self.pages = torch.full((users, pages_of_user), -1, dtype=torch.int32)

    def _batch(self, counts):
        """Offsets, lengths and page table on the GPU; pages are given out as histories grow."""
        for u, length in enumerate(self.lengths):
            for p in range(-(-length // self.page_size)):
                if self.pages[u, p] < 0:
                    self.pages[u, p] = self.free.pop()
        offsets = torch.tensor([0] + counts).cumsum(0)
        return [t.to(self.model.device) for t in (offsets, torch.tensor(self.lengths), self.pages)]

    def _attend(self, q, batch, counts, causal):
        m, out = self.model, torch.empty_like(q)
        sizes = len(counts), q.shape[0], m.q_heads, m.kv_heads, m.d, max(counts), max(self.lengths)
        workspace = torch.empty(sdi.dlrm_kv_attn_workspace_size(*sizes), dtype=torch.uint8, device=m.device)
        sdi.dlrm_kv_attn_fwd(q, *batch, self.k, self.v, out, m.d ** -0.5, workspace, max(counts), max(self.lengths),
                             causal=causal, err_flag=m.err)
        return out

    def append(self, counts, items):
        """Stores ``counts[u]`` new events of each user; returns what each gathers from those up to itself."""
        m = self.model
        self.lengths = [n + c for n, c in zip(self.lengths, counts)]
        batch = self._batch(counts)
        q, k, v = m.heads(items)
        q_out = torch.empty(q.shape, dtype=m.dtype, device=m.device)
        sdi.dlrm_kv_append(k, v, *batch, self.k, self.v, k_weight=m.k_weight, eps=m.eps, rope=m.rope, q=q,
                           q_weight=m.q_weight, q_out=q_out, err_flag=m.err)
        return self._attend(q_out, batch, counts, True)

    def candidates(self, counts, items):
        """What ``counts[u]`` candidate items gather from each user's whole history, as the next event would."""
        m = self.model
        batch = self._batch(counts)
        q = m.heads(items)[0]
        at = torch.tensor(self.lengths).repeat_interleave(torch.tensor(counts)).to(m.device)
        q_out = torch.empty(q.shape, dtype=m.dtype, device=m.device)
        sdi.dlrm_qk_norm_rope_fwd(q, None, m.q_weight, None, m.eps, m.rope, at, q_out, None)
        return self._attend(q_out, batch, counts, False)


def serve(model, users=5, seed=1):
    """Stores histories, an event more for some, then scores candidates; returns
    the histories, their items, the candidates' counts and items, what they
    gather and the interaction's output."""
    g = torch.Generator().manual_seed(seed)
    pick = lambda n: torch.randint(model.table.shape[0], (n,), generator=g).to(model.device)
    store, past = Histories(model, users), [[] for _ in range(users)]
    for counts in ([40 + 37 * u for u in range(users)], [1 - u % 2 for u in range(users)], [1] * users):
        items = pick(sum(counts))
        store.append(counts, items)
        for mine, new in zip(past, items.split(counts)):
            mine.append(new)
    counts = [1 + 13 * u for u in range(users)]
    items = pick(sum(counts))
    gathered = store.candidates(counts, items)
    # beside the candidate's own vector: its user's pooled recent items, and what it gathered
    n, width = items.numel(), model.table.shape[1]
    vectors = torch.empty((n, 2, width), device=model.device)
    recent = torch.cat([torch.cat(mine)[-20:] for mine in past])
    bags = torch.empty((users, 1, width), device=model.device)
    sdi.dlrm_emb_bag_fwd([model.table], torch.arange(0, 20 * users + 1, 20, device=model.device), recent, users, bags,
                         err_flag=model.err)
    vectors[:, 0] = bags[:, 0].repeat_interleave(torch.tensor(counts, device=model.device), 0)
    vectors[:, 1] = gathered.flatten(1).float() @ model.back
    own, y = model.table[items], torch.empty((n, width + sdi.dlrm_num_pairs(2, False)), device=model.device)
    sdi.dlrm_interact_fwd(own, vectors, False, y)
    status = sdi.dlrm_read_error(model.err)
    if status != 0:
        raise RuntimeError(f"device error flag: {sdi.status_string(status)}")
    return store, [torch.cat(mine) for mine in past], counts, items, gathered, y


def train(model, tokens=96, steps=30, rate=3.0, seed=2):
    """Fits the norms' weights so that the attention scores of a chunk of events
    come near given ones; returns the losses."""
    g = torch.Generator().manual_seed(seed)
    items = torch.randint(model.table.shape[0], (tokens,), generator=g).to(model.device)
    q, k, _ = (t.float().contiguous() for t in model.heads(items))
    at = torch.arange(tokens, device=model.device)
    group = model.q_heads // model.kv_heads

    def scores(q_weight, k_weight):
        qn, kn = NormRope.apply(q, k, q_weight, k_weight, model.eps, model.rope, at)
        return torch.einsum("ihd,jhd->hij", qn, kn.repeat_interleave(group, 1)) * model.d ** -0.5

    target = scores(model.q_weight, model.k_weight)
    weights = [torch.ones(model.d, device=model.device, requires_grad=True) for _ in range(2)]
    losses = []
    for _ in range(steps):
        loss = (scores(*weights) - target).square().mean()
        losses.append(loss.item())
        for w, dw in zip(weights, torch.autograd.grad(loss, weights)):
            with torch.no_grad():
                w -= rate * dw
    return losses


def main():
    model = HistoryModel()
    store, past, counts, items, gathered, y = serve(model)
    print(f"{len(past)} users with {store.lengths} stored events; {items.numel()} candidates scored, "
          f"interaction output {tuple(y.shape)}")
    losses = train(model)
    print(f"norm weights fitted: loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
