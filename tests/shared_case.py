"""Batches whose sequences share prefixes, for the tests, on the CPU: as forks of prompts leave them."""
import torch

from paged_case import Case, quantize


class Shared(Case):
    """groups of sequences [(prefix, [(own tokens, tokens of the call), ...]), ...]: the prefix's whole pages are the
    same for all, the page that it ends in is each one's own copy, with other tokens behind."""

    def __init__(self, groups, seed=0, before=(), **kw):
        seqs = list(before) + [(p + own, n) for p, rest in groups for own, n in rest]
        super().__init__(n=[n for _, n in seqs], kv=[k for k, _ in seqs], seed=seed, **kw)
        self.groups, self.prefix = [len(before)], [p for p, _ in groups]
        for g, (p, rest) in enumerate(groups):
            first = self.groups[-1]
            self.groups.append(first + len(rest))
            whole = p // self.page
            for b in range(first + 1, self.groups[-1]):
                self.table[b, :whole] = self.table[first, :whole]
                if p % self.page:
                    a, e = int(self.table[first, whole]), int(self.table[b, whole])
                    for x in (self.K8, self.V8, self.sk, self.sv):
                        x[e, :, :p % self.page] = x[a, :, :p % self.page]

    def shared_args(self, device):
        return tuple(torch.tensor(x, dtype=torch.int32, device=device) for x in (self.groups, self.prefix))

    def most(self):
        return max([sum(self.n[a:b]) for a, b in zip(self.groups, self.groups[1:])], default=0)


def values(shape, mul, seed):
    """Quantized rows of N(0, mul^2)."""
    return quantize((torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * mul).to(torch.bfloat16))
