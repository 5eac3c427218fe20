"""Inputs of the latent-attention tests and their results in 64 bits, from the
formulas alone (torch float64, no code of the package)."""
import torch

ROPE = 64


def normal(seed, *shape, std=1.0, device="cuda"):
    gen = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device=device) * std).to(torch.bfloat16)


class Paged:
    """A paged cache: request b holds contexts[b] + drafts[b] tokens, its pages
    spread over the pool in random order.  Entries of the table past a
    request's pages, the pages no request holds and the slots past a length
    are poison."""

    def __init__(self, contexts, drafts, latent, page_size, seed=0, spare=3, poison=float("nan"),
                 keys=None):
        width = latent + ROPE
        self.latent, self.page_size = latent, page_size
        self.contexts, self.drafts = list(contexts), list(drafts)
        self.lengths_list = [c + d for c, d in zip(contexts, drafts)]
        need = [-(-n // page_size) for n in self.lengths_list]
        pool = sum(need) + spare
        host = torch.Generator().manual_seed(seed)
        order = torch.randperm(pool, generator=host).tolist()
        self.cache = torch.full((pool, page_size, width), poison, dtype=torch.bfloat16,
                                device="cuda")
        table = torch.full((len(need), max(max(need), 1)), -7, dtype=torch.int32)
        self.tokens = []
        for b, n in enumerate(self.lengths_list):
            rows = normal(seed * 1000 + b, n, width) if keys is None else keys(b, n, width)
            self.tokens.append(rows)
            for i in range(need[b]):
                page = order.pop()
                table[b, i] = page
                part = rows[i * page_size:(i + 1) * page_size]
                self.cache[page, :part.shape[0]] = part
        self.table = table.cuda()
        self.lengths = torch.tensor(self.lengths_list, dtype=torch.int32, device="cuda")
        begin = [0]
        for d in drafts:
            begin.append(begin[-1] + d)
        self.rows = begin[-1]
        self.begin_list = begin
        self.begin = torch.tensor(begin, dtype=torch.int32, device="cuda")

    def random_tree(self, seed):
        """A random forest over each request's drafts, as ancestor masks."""
        host = torch.Generator().manual_seed(seed)
        masks = []
        for d in self.drafts:
            sees = []
            for j in range(d):
                up = int(torch.randint(-1, j, (1,), generator=host)) if j else -1
                sees.append((sees[up] if up >= 0 else 0) | 1 << j)
            masks += sees
        return masks

    def expected(self, q, scale, masks=None):
        """(out, weight): the attention in float64 and, for the tolerance, the
        same weights over the latents' magnitudes."""
        rows, heads = q.shape[0], q.shape[1]
        out = torch.zeros(rows, heads, self.latent, dtype=torch.float64, device="cuda")
        weight = torch.zeros_like(out)
        for b, tokens in enumerate(self.tokens):
            c = self.contexts[b]
            for t in range(self.drafts[b]):
                row = self.begin_list[b] + t
                drafts = [j for j in range(self.drafts[b])
                          if (j <= t if masks is None else j < 64 and masks[row] >> j & 1)]
                keep = list(range(c)) + [c + j for j in drafts]
                if not keep:
                    continue
                mine = tokens[torch.tensor(keep, device="cuda")].double()
                p = torch.softmax(q[row].double() @ mine.t() * scale, -1)
                out[row] = p @ mine[:, :self.latent]
                weight[row] = p @ mine[:, :self.latent].abs()
        return out, weight


def masks_tensor(masks):
    """64-bit masks as the int64 tensor the call takes."""
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64,
                        device="cuda")
