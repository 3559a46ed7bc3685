"""Paged caches for the tests: pools, tables and new tokens of ragged sequences, and the plain
reading of them."""
import torch


class Paged:
    """Sequences of lens cached and news new positions over a pool in which every place that is
    nobody's holds `stale`."""

    def __init__(self, lens, news, Hkv, d, page, seed, order="places", stale=float("nan"), spare=3, extra=0):
        from bit_moe_expert_route_gb300 import ops
        g = torch.Generator(device="cuda").manual_seed(seed)
        host = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.lens_list, self.news, self.page, self.Hkv, self.d = list(lens), list(news), page, Hkv, d
        need = [-(-(a + n) // page) for a, n in zip(lens, news)]
        n_pages = sum(need) + spare
        ids = torch.randperm(n_pages, generator=host).tolist()
        table = torch.full((B, max(need + [1]) + extra), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
            at += n
        self.starts_list = [0]
        for n in news:
            self.starts_list.append(self.starts_list[-1] + n)
        self.N = self.starts_list[-1]

        def pool():
            if order == "places":    # [page, place, head]
                return torch.empty(n_pages, page, Hkv, d, dtype=torch.bfloat16, device="cuda"), None
            if order == "heads":     # [page, head, place]
                return torch.empty(n_pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda").transpose(1, 2), None
            both = torch.empty(n_pages, page, 2, Hkv, d, dtype=torch.bfloat16, device="cuda")  # K and V side by side
            return both[:, :, 0], both[:, :, 1]
        k, v = pool()
        if v is None:
            v, _ = pool()
        k.fill_(stale), v.fill_(stale)
        self.cache = ops.PagedCache(k, v, table.cuda())
        self.table = table
        self.starts = torch.tensor(self.starts_list, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.g = g

    def normal(self, *shape, std=1.0):
        return torch.randn(*shape, generator=self.g, device="cuda").mul(std).bfloat16()

    def places(self, b, positions):
        """(pages, places) of a sequence's positions, on the GPU."""
        p = torch.as_tensor(positions, dtype=torch.int64)
        return self.table[b].long()[p // self.page].cuda(), (p % self.page).cuda()

    def fill(self):
        """Every position, cached and new, gets keys and values."""
        for b, (a, n) in enumerate(zip(self.lens_list, self.news)):
            if a + n:
                to = self.places(b, torch.arange(a + n))
                for t in self.cache[:2]:
                    t[to] = self.normal(a + n, self.Hkv, self.d)
        return self

    def read(self, b):
        """K and V of a sequence, cached and new, [positions, Hkv, d]."""
        to = self.places(b, torch.arange(self.lens_list[b] + self.news[b]))
        return self.cache.k_pages[to], self.cache.v_pages[to]


def random_tree(news, seed):
    """Masks of random trees (int64, on the GPU), each token following an earlier one or the cache."""
    from bit_moe_expert_route_gb300 import ops
    host = torch.Generator().manual_seed(seed)
    masks = []
    for n in news:
        up = [int(torch.randint(-1, i, (1,), generator=host)) if i else -1 for i in range(n)]
        masks.append(ops.tree_masks(up)[0])
    return torch.cat(masks + [torch.zeros(0, dtype=torch.int64)]).cuda()
