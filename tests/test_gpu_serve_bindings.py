"""The plain bindings of the packed and paged calls against the classes that
own their workspaces: the same buffers, bit for bit."""
import pytest

from int4_quantized_attention_b200 import api, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

D, F16 = 128, torch.float16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return api.lib()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(F16)


def zeros(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("hq", [4, 64])
def test_packed(hq):
    cu, n = ints([0, 700, 701, 1300]), 1300
    q, k, v = rand(1, n, hq, D), rand(2, n, hq // 2, D), rand(3, n, hq // 2, D)
    want, wl = api.PackedAttention().forward(q, k, v, cu, cu, return_lse=True)
    p = api.Packed(3, hq, hq // 2, D, api.DTYPE_FP16, 1, n, n, 0.0, hq * D, D, *([hq // 2 * D, D] * 2), hq * D, D)
    ws, o, lse = zeros(api.packed_workspace_bytes(p)), torch.empty_like(q), torch.empty_like(wl)
    api.packed_attention_fwd(p, q, k, v, cu, cu, o, lse, ws)
    api.check_device_error(ws)
    assert torch.equal(o, want) and torch.equal(lse, wl)


def test_cache():
    args = (2, 40, 16, 2, 6, 9)
    a = api.PagedCache(*args, pool=torch.zeros(2, 2, 40, 2, 16, D, dtype=F16, device="cuda"))
    p = api.CacheProblem(2, 40, 16, 2, D, api.DTYPE_FP16, 6, 9)
    assert api.cache_validate(p) == api.RA_OK
    pool, state = zeros(api.cache_pool_bytes(p)), zeros(api.cache_state_bytes(p))
    c, ws = api.cache_bind(p, pool, state), zeros(api.cache_workspace_bytes(p))
    api.cache_init(p, c)
    rows, new, cu = ints([0, 3]), ints([40, 17]), ints([0, 40, 57])
    k, v, q = rand(1, 57, 2, D), rand(2, 57, 2, D), rand(3, 4, 4, D)
    a.extend(rows, new)
    api.cache_extend(p, c, rows, new, ws)
    for layer in range(2):
        a.write(layer, rows, k, v, cu_new=cu)
        api.cache_write(p, c, layer, rows, cu, k, v, ws)
    a.fork(ints([0, 0, 3]), ints([1, 2, 4]))
    api.cache_fork(p, c, ints([0, 0, 3]), ints([1, 2, 4]), ws)
    a.extend(ints([1, 2]), ints([1, 1]))
    api.cache_extend(p, c, ints([1, 2]), ints([1, 1]), ws)
    a.write(1, ints([1, 2]), k[:2], v[:2])
    api.cache_write(p, c, 1, ints([1, 2]), None, k[:2], v[:2], ws)
    a.free(ints([0]))
    api.cache_free(p, c, ints([0]), ws)
    a.compact()
    api.cache_compact(p, c, ws)
    seqs = ints([1, 2, 3, 4])
    want, wl = a.attention(1, q, seqs, return_lse=True)
    at = api.CacheAttn(4, 4, 4, 1, 0, 0.0, 4 * D, D, 4 * D, D)
    aws, o, lse = zeros(api.cache_attention_workspace_bytes(p, at)), torch.empty_like(q), torch.empty_like(wl)
    api.cache_attention_fwd(p, c, at, q, seqs, None, o, lse, aws)
    a.check()
    api.check_device_error(ws)
    api.check_device_error(aws)
    assert torch.equal(o, want) and torch.equal(lse, wl)
    # words between refs, lens and table, whose last bytes are padding, belong to nobody
    for x, n in (("refs", 40), ("lens", 6), ("table", 54)):
        off = getattr(c, x) - state.data_ptr()
        assert torch.equal(state[off:off + 4 * n].view(torch.int32), getattr(a, x).reshape(-1)), x
    assert torch.equal(pool.view(torch.int16), a.pool.view(-1).view(torch.int16))
