"""The 4-bit cache beyond 4 GB a plane: every operator at its far end."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from . import kv4_reference as ref  # noqa: E402
from .test_gpu_kv4 import DEV, check, dk, i32, normal, query  # noqa: E402,F401

pytestmark = pytest.mark.gpu

PAGE = 64


@pytest.mark.parametrize("heads,dim", [(8, 128), (5, 128), (4, 64)])
def test_slots_whose_bytes_lie_beyond_32_bits(dk, heads, dim):  # noqa: F811
    rng = np.random.default_rng(heads)
    pages = (2 ** 32 // (heads * dim // 2) + 2 ** 16) // PAGE
    last = 24  # pages in use, the plane's last ones
    cache = dk.Kv4Cache.allocate(pages, PAGE, heads, dim, DEV)
    first = pages - last
    assert (first * PAGE) * heads * dim // 2 >= 2 ** 32 - 2 ** 24
    assert ((pages - 1) * PAGE) * heads * dim // 2 > 2 ** 32
    # append and read
    n = last * PAGE
    k, v = normal(rng, n, heads, dim), normal(rng, n, heads, dim)
    slots = torch.arange(first * PAGE, pages * PAGE, device=DEV)
    dk.kv4_append(cache, *[torch.from_numpy(x).float().to(DEV) for x in (k, v)], slots)
    planes = []
    for x in (k, v):
        codes, scales = ref.encode(x.astype(np.float32))
        planes.append((ref.pack(codes).reshape(last, PAGE, heads, -1),
                       scales.astype(np.uint8).reshape(last, PAGE, heads, -1)))
    host = (planes[0][0], planes[1][0], planes[0][1], planes[1][1])
    got = dk.kv4_read(cache, slots, dtype=torch.float32)
    for i in range(2):
        want = ref.decode(host[i], host[2 + i]).reshape(n, heads, dim)
        assert np.array_equal(got[i].double().cpu().numpy(), want)
    for plane in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales):
        assert not plane[:first].any()

    # attention: a few rows (slices), a wide table (shares), ids and a range
    rows, width = 4, 20
    lens = np.array([1280, 1000, 33, 641])
    near = np.stack([rng.permutation(last)[:width] for _ in range(rows)])
    q, values = query(rng, rows, heads * 2, dim, "bf16")
    ids = rng.integers(0, 1280, (rows, 700))
    for wide in (width, 1500):
        table = np.full((rows, wide), -1)
        table[:, :width] = near
        for chosen in (None, ids):
            named = {} if chosen is None else {"ids": i32(chosen)}
            out, lse = dk.kv4_attention(cache, q, i32(np.where(table < 0, -1, table + first)),
                                        i32(lens), **named)
            small = dk.Kv4Cache(*[torch.from_numpy(p).to(DEV) for p in host])
            want = dk.kv4_attention(small, q, i32(table), i32(lens), **named)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    check(dk, small, host, q, values, "bf16", near, lens)

    # eviction from the far end into its last pages
    w = torch.from_numpy(rng.random((1, 1280))).float().to(DEV)
    kept, _, _ = dk.kv4_evict(cache, i32(np.arange(20)[None] + first), i32([1280]), w,
                              i32([[pages - 4, pages - 2]]), 2 * PAGE)
    kept = kept[0].cpu().numpy()
    for name, p in zip(("k_codes", "v_codes", "k_scales", "v_scales"), host):
        moved = getattr(cache, name)[[pages - 4, pages - 2]].flatten(0, 1).cpu().numpy()
        assert np.array_equal(moved, p.reshape(n, heads, -1)[kept])
