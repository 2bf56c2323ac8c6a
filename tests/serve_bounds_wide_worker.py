"""Worker of tests/test_gpu_serve_bounds_wide.py: the page operations and the
attention over a cache on whichever build RA_LIBRARY selects, with long lists,
writes of one and of many tokens, forks, and more rows than a query tile holds.

    python tests/serve_bounds_wide_worker.py OUT.npz
"""
import sys

from serve_bounds_worker import D, api, ints, np, poison_workspaces, poisoned, status, torch

BF16 = torch.bfloat16


def main(path):
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)   # noqa: E731
    res = {}
    for page in (16, 128):
        c = api.PagedCache(1, 900, page, 1, 300, 6, dtype=BF16, pool=poisoned(2, 1, 900, 1, page, D, dtype=BF16))
        poison_workspaces(c)
        every = list(range(150))
        c.extend(ints(every), ints([page + 1 + i % page for i in every]))
        for count in (1, page):
            k, v = rand(150 * count, 1, D), rand(150 * count, 1, D)
            c.write(0, ints(every), k, v, cu_new=None if count == 1 else ints([count * i for i in range(151)]))
        c.fork(ints(every), ints([150 + i for i in every]))
        c.free(ints(every[::2]))
        c.compact()
        k = rand(2 * page + 1, 1, D)
        c.extend(ints([0]), ints([2 * page + 1]))
        c.write(0, ints([0]), k, k, cu_new=ints([0, 2 * page + 1]))
        q = rand(600, 8, D)
        for cu in (None, ints([2 * i for i in range(301)])):
            rows = 300 if cu is None else 600
            out = poisoned(rows, 8, D, dtype=BF16)
            c.attention(0, q[:rows], ints(list(range(300))), cu_q=cu, out=out)
            poison_workspaces(c)
            res[f"{page}/{rows}"] = out.view(torch.int16)
        res[f"{page}/pool"], res[f"{page}/state"] = c.pool.view(torch.int16), c.state
        res[f"{page}/status"] = status(c)
    np.savez(path, **{k: v.cpu().numpy() if torch.is_tensor(v) else v for k, v in res.items()})


if __name__ == "__main__":
    main(sys.argv[1])
