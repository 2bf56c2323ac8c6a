"""Worker of tests/test_gpu_serve_bounds.py: the packed and paged calls of
whichever build RA_LIBRARY selects, on cases with ragged ends, outputs and
workspaces filled with 0x77 first; saves the outputs and statuses.

    python tests/serve_bounds_worker.py OUT.npz
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

from int4_quantized_attention_b200 import api  # noqa: E402

D = 128


def poisoned(*shape, dtype=torch.float16):
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    return torch.full((n,), 0x77, dtype=torch.uint8, device="cuda").view(dtype).view(*shape)


def poison_workspaces(op):
    op._ws.current()[256:] = 0x77
    if hasattr(op, "_work"):
        op._work[256:] = 0x77


def status(op):
    try:
        op.check()
        return api.RA_OK
    except api.RotateAttnError as e:
        print(e)
        return e.status


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def main(path):
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s, t=torch.float16: torch.randn(*s, generator=g, device="cuda").to(t)   # noqa: E731
    res = {}
    op = api.PackedAttention()
    for name, lens, past, hq, hkv, t in (("few", [1, 77, 130, 0, 5], 300, 10, 2, torch.float16),
                                         ("whole", [300, 129, 700, 1], 40, 48, 48, torch.bfloat16)):
        cq, ck = np.cumsum([0] + lens).tolist(), np.cumsum([0] + [n + past for n in lens]).tolist()
        q, k, v = rand(cq[-1], hq, D, t=t), rand(ck[-1], hkv, D, t=t), rand(ck[-1], hkv, D, t=t)
        out, lse = poisoned(cq[-1] + 3, hq, D, dtype=t), poisoned(cq[-1] + 3, hq, dtype=torch.float32)
        qq = torch.cat([q, q[:3]])
        for _ in range(2):
            op.forward(qq, k, v, ints(cq), ints(ck), out=out, lse=lse)
            poison_workspaces(op)
        res[name + "/o"], res[name + "/lse"] = out.view(torch.int16), lse.view(torch.int32)
        res[name + "/status"] = status(op)
    for page in (16, 128):
        n = 6
        pool = poisoned(2, 2, 90, 2, page, D)
        c = api.PagedCache(2, 90, page, 2, n + 1, 12, pool=pool)
        poison_workspaces(c)
        c.extend(ints([n]), ints([2 * page + 3]))
        k, v = rand(2 * page + 3, 2, D), rand(2 * page + 3, 2, D)
        for layer in range(2):
            c.write(layer, ints([n]), k, v, cu_new=ints([0, 2 * page + 3]))
        c.fork(ints([n] * n), ints(list(range(n))))
        new = [1, 5, page, 3 * page + 1, 2, 40]
        c.extend(ints(list(range(n))), ints(new))
        cu = np.cumsum([0] + new).tolist()
        k, v, q = rand(cu[-1], 2, D), rand(cu[-1], 2, D), rand(cu[-1], 10, D)
        for layer in range(2):
            c.write(layer, ints(list(range(n))), k, v, cu_new=ints(cu))
        c.free(ints([n, 2]))
        c.compact()
        for shared in (0, 2 * page):
            for single in (False, True):
                rows = n if single else cu[-1]
                out, lse = poisoned(rows, 10, D), poisoned(rows, 10, dtype=torch.float32)
                c.attention(1, q[:rows], ints(list(range(n))), cu_q=None if single else ints(cu), shared=shared, out=out,
                            lse=lse)
                poison_workspaces(c)
                res[f"{page}/{shared}/{single}/o"], res[f"{page}/{shared}/{single}/lse"] = out.view(torch.int16), lse.view(torch.int32)
        res[f"{page}/state"], res[f"{page}/pool"] = c.state, c.pool.view(torch.int16)
        res[f"{page}/status"] = status(c)
    np.savez(path, **{k: v.cpu().numpy() if torch.is_tensor(v) else v for k, v in res.items()})


if __name__ == "__main__":
    main(sys.argv[1])
