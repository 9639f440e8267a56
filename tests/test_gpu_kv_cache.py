"""GPU: page assignment, the cache write and the accepted path's move against
their definitions (tests/kv_reference.py): whole numbers and codes are equal."""
import numpy as np
import pytest
import torch

import quantization_amax_reduce_b200 as qar
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def dev32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


class DevicePool:
    def __init__(self, p: ref.Pool):
        self.page = p.page
        self.tables = dev32(p.tables)
        self.owned = dev32(p.owned)
        free = np.full(p.num_pages, -7, dtype=np.int32)
        free[:len(p.free)] = p.free
        self.free = dev32(free)
        self.pool = dev32([len(p.free), 0])
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def assign(self, seq, new, max_tokens, **kw):
        got = qar.kv_assign_pages(dev32(seq), dev32(new), self.tables, self.owned, self.free,
                                  self.pool, self.page, max_tokens, error=self.err, **kw)
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in got]

    def check(self, p: ref.Pool):
        assert self.pool.tolist() == [len(p.free), 0]
        assert self.free[:len(p.free)].tolist() == p.free
        assert self.owned.tolist() == list(p.owned)
        assert np.array_equal(self.tables.cpu().numpy(), p.tables)


@pytest.mark.parametrize("rows,page,longest", [
    (1, 16, 100), (3, 8, 500), (64, 16, 300), (513, 32, 90), (2000, 16, 60), (5000, 64, 200),
    (7, 1024, 9000),
])
def test_assign_pages_over_many_steps(rows, page, longest):
    r = np.random.Generator(np.random.PCG64(rows))
    width = -(-longest // page)
    num = max(4, int(0.7 * rows * width))
    p = ref.Pool(rows, width, num, page, r.permutation(num))
    d = DevicePool(p)
    seq = np.zeros(rows, dtype=np.int64)
    refused = 0
    for step in range(7):
        # requests grow, shrink (a rejected draft), end and start in one step
        new = r.integers(0, max(2, longest // 4), rows)
        base = np.where(r.random(rows) < 0.2, 0, np.where(r.random(rows) < 0.3, seq // 2, seq))
        want = np.minimum(base + new, longest)
        new = want - np.minimum(base, want)
        cap = int(new.sum()) + int(r.integers(0, 50))
        expect = p.assign(want, new, cap)
        got = d.assign(want, new, cap)
        if expect is None:
            refused += 1
            assert qar.read_error_word(d.err) == 7
            assert (got[0] == 0).all() and (got[1] == -1).all() and (got[2] == 0).all()
        else:
            assert qar.read_error_word(d.err) == 0
            for a, b in zip(got, expect):
                assert np.array_equal(a, b)
            seq = want
        d.check(p)
    assert refused < 7


def test_assign_pages_growth_and_release_restore_the_free_list():
    r = np.random.Generator(np.random.PCG64(9))
    p = ref.Pool(300, 40, 12000, 16, r.permutation(12000))
    d = DevicePool(p)
    before = d.free.clone()
    lens = r.integers(1, 640, 300)
    d.assign(lens, lens, int(lens.sum()))
    d.assign(lens * 0, lens * 0, 0)
    assert torch.equal(d.free, before) and d.pool.tolist() == [12000, 0]
    assert qar.read_error_word(d.err) == 0


@pytest.mark.parametrize("why,seq,new,tokens,status", [
    ("new beyond the length", [5, 3], [1, 4], 64, 6),
    ("negative new", [5, 3], [-1, 3], 64, 6),
    ("longer than the table", [5, 16 * 4 + 1], [1, 1], 64, 6),
    ("more tokens than max_tokens", [40, 40], [40, 40], 79, 6),
    ("too few free pages", [60, 60], [1, 1], 64, 7),
])
def test_assign_pages_refused_steps_change_nothing(why, seq, new, tokens, status):
    p = ref.Pool(2, 4, 6, 16)
    assert p.assign([5, 3], [5, 3], 8) is not None
    d = DevicePool(p)
    got = d.assign(seq, new, tokens)
    assert qar.read_error_word(d.err) == status
    assert (got[0] == 0).all() and (got[1] == -1).all()
    d.check(p)
    # and the pool still works
    expect = p.assign([20, 3], [15, 0], 15)
    for a, b in zip(d.assign([20, 3], [15, 0], 15), expect):
        assert np.array_equal(a, b)


def test_assign_pages_bad_page_ids_are_reported_and_not_followed():
    p = ref.Pool(2, 4, 8, 16)
    p.assign([20, 20], [20, 20], 40)
    d = DevicePool(p)
    d.tables[0, 1] = 99                                # in the part that row 0 writes to
    d.free[int(d.pool[0]) - 1] = -5                    # the next page to be taken
    got = d.assign([22, 40], [2, 20], 22)
    assert qar.read_error_word(d.err) == 7
    slots = got[1]
    assert (slots[:2] == -1).all()                     # row 0: page 99
    assert (slots[2:2 + 12] >= 0).all()                # row 1: positions 20..31
    assert (slots[14:] == -1).all()                    # row 1: the bad new page


@pytest.mark.parametrize("bad", [99, -1, -(2 ** 31)])
def test_assign_pages_bad_page_ids_given_back_are_reported(bad):
    """A page id outside the pool that a request gives back sets the error at
    once, not in the step of the request that takes it next."""
    p = ref.Pool(3, 4, 10, 16)
    p.assign([20, 40, 5], [20, 40, 5], 65)
    d = DevicePool(p)
    d.tables[1, 1] = bad
    d.assign([20, 10, 5], [0, 0, 0], 0)               # row 1 gives back its second and third
    assert qar.read_error_word(d.err) == 7
    p.tables[1, 1] = bad
    p.assign([20, 10, 5], [0, 0, 0], 0)
    d.check(p)                                        # (the list keeps its order and length)
    # one that is passed on to a row that grows in the same step is not followed
    q = ref.Pool(2, 4, 10, 16)
    q.assign([40, 5], [40, 5], 45)
    d = DevicePool(q)
    d.tables[0, 1] = bad
    _, slots, _ = d.assign([10, 40], [0, 35], 35)
    assert qar.read_error_word(d.err) == 7
    second = int(d.tables[0, 2])
    assert d.tables[1].tolist()[:3] == [int(q.tables[1, 0]), -1, second]
    assert (slots[:11] >= 0).all() and (slots[11:27] == -1).all()
    assert (slots[27:] // 16 == second).all()


def test_assign_pages_captured_at_a_fixed_size():
    """A step captured once, replayed over changing lengths."""
    r = np.random.Generator(np.random.PCG64(11))
    rows, page, cap = 40, 16, 256
    p = ref.Pool(rows, 64, 1500, page, r.permutation(1500))
    d = DevicePool(p)
    seq, new = dev32(np.zeros(rows)), dev32(np.zeros(rows))
    out = (torch.empty(rows + 1, dtype=torch.int32, device=DEV),
           torch.empty(cap, dtype=torch.int64, device=DEV),
           torch.empty(cap, dtype=torch.int32, device=DEV))
    call = lambda: qar.kv_assign_pages(seq, new, d.tables, d.owned, d.free, d.pool, page, cap,  # noqa: E731
                                       out=out, error=d.err)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    have = np.zeros(rows, dtype=np.int64)
    for _ in range(5):
        add = r.integers(0, 7, rows)
        have = have + add
        seq.copy_(dev32(have))
        new.copy_(dev32(add))
        expect = p.assign(have, add, cap)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, expect):
            assert np.array_equal(a.cpu().numpy(), b)
        d.check(p)
    assert qar.read_error_word(d.err) == 0


def test_assign_pages_of_two_threads_with_many_rows():
    """Both calls need more shared memory than a launch gets unasked, in
    different amounts: neither may take the other's away."""
    import threading
    failed = []

    def work(rows):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                p = ref.Pool(rows, 2, 2 * rows, 16)
                d = DevicePool(p)
                seq = np.full(rows, 20)
                new = np.zeros(rows, dtype=np.int64)
                args = (dev32(seq), dev32(new), d.tables, d.owned, d.free, d.pool, 16, 0)
                for _ in range(400):
                    qar.kv_assign_pages(*args, error=d.err)
                stream.synchronize()
                assert qar.read_error_word(d.err) == 0
                p.assign(seq, new, 0)
                d.check(p)
        except Exception as e:   # noqa: BLE001 (handed to the test)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(rows,)) for rows in (16384, 4500)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_assign_pages_just_below_the_shared_memory_of_a_plain_launch():
    """Row counts whose prefix sums alone fit 48 KB of shared memory, but not
    beside the kernel's own, in a process that made no larger call before."""
    code = """if True:
        import numpy as np, torch
        from tests import kv_reference as ref
        from tests.test_gpu_kv_cache import DevicePool, qar
        for rows in (4061, 4062, 4080, 4095, 4096):
            p = ref.Pool(rows, 2, 2 * rows, 16)
            d = DevicePool(p)
            seq, new = np.full(rows, 20), np.full(rows, 3)
            want, got = p.assign(seq, new, 3 * rows), d.assign(seq, new, 3 * rows)
            assert all(np.array_equal(g, w) for g, w in zip(got, want)), rows
            assert qar.read_error_word(d.err) == 0
            d.check(p)
    """
    import subprocess
    import sys
    from tests.conftest import ROOT
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]


# ---------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------

def codes_of(x, scale):
    """E4M3 codes of fl32(x * scale), NaN as 0x7F whatever its sign."""
    y = (x.float() * scale).clamp(-448, 448)
    c = y.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(torch.isnan(y), torch.full_like(c, 0x7F), c)


def cache_views(pages, page, heads, dtype, layout):
    """K and V caches [pages, page, heads, 128] of one layout, full of a marker."""
    if layout == "token":
        base = torch.empty(2, pages, page, heads, 128, dtype=dtype, device=DEV)
        k, v = base[0], base[1]
    elif layout == "head":
        base = torch.empty(2, pages, heads, page, 128, dtype=dtype, device=DEV)
        k, v = base[0].transpose(1, 2), base[1].transpose(1, 2)
    else:      # K and V of a page side by side, and rows wider than the heads
        base = torch.empty(pages, 2, page, heads + 1, 128, dtype=dtype, device=DEV)
        k, v = base[:, 0, :, :heads], base[:, 1, :, :heads]
    base.fill_(3)
    return base, k, v


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("layout", ["token", "head", "interleaved"])
@pytest.mark.parametrize("tokens,heads,page", [(1, 1, 16), (7, 5, 8), (300, 8, 64), (65, 40, 1024)])
def test_write(tokens, heads, page, layout, fp8):
    g = torch.Generator().manual_seed(tokens)
    pages = -(-tokens // page) + 2
    base, kc, vc = cache_views(pages, page, heads, torch.uint8 if fp8 else torch.bfloat16, layout)
    before = base.clone()
    qkv = (torch.randn(tokens, 3, heads, 128, generator=g) * 40).to(torch.bfloat16)
    flat = qkv.view(-1)
    flat[::97], flat[5::101], flat[7::89] = float("inf"), float("nan"), -0.0
    flat[3::83] = -float("nan")
    qkv = qkv.to(DEV)
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    if tokens > 2:
        slots[1] = -1
        slots[2] = -(2 ** 40)
    scale = torch.tensor([1.0, 448 / 210.0, 448 / 33.0], device=DEV) if fp8 else None
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qar.kv_write(qkv[:, 1], qkv[:, 2], slots.to(DEV), kc, vc, scale, error=err)
    torch.cuda.synchronize()
    assert qar.read_error_word(err) == 0
    live = slots >= 0
    for t, cache in ((1, kc), (2, vc)):
        x = qkv[:, t][live.to(DEV)]
        want = codes_of(x, scale[t]) if fp8 else x
        s = slots[live].to(DEV)
        got = cache[s // page, s % page]
        assert torch.equal(got.view(torch.uint8), want.contiguous().view(torch.uint8))
        cache[s // page, s % page] = 3
    assert torch.equal(base.view(torch.uint8), before.view(torch.uint8))   # nothing else


def test_write_slots_beyond_the_cache_are_reported_and_skipped():
    base, kc, vc = cache_views(2, 16, 2, torch.bfloat16, "token")
    x = torch.randn(4, 2, 128, device=DEV).to(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qar.kv_write(x, x, torch.tensor([32, 5, 2 ** 62, 31], device=DEV), kc, vc, error=err)
    torch.cuda.synchronize()
    assert qar.read_error_word(err) == 7
    assert torch.equal(kc[0, 5], x[1]) and torch.equal(vc[1, 15], x[3])
    rest = kc.reshape(32, 2, 128)[[i for i in range(32) if i not in (5, 31)]]
    assert (rest == 3).all()


def test_write_and_attend_beyond_4_gib():
    """Offsets past 32 bits: the last pages of a cache of 2 x 5 GiB."""
    page, heads = 256, 8
    pages = (5 << 30) // (page * heads * 128)
    kc = torch.zeros(pages, page, heads, 128, dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    n = 300
    k = torch.randn(n, heads, 128, device=DEV).to(torch.bfloat16)
    v = torch.randn(n, heads, 128, device=DEV).to(torch.bfloat16)
    table = torch.tensor([[pages - 1, 7]], dtype=torch.int32, device=DEV)
    t = torch.arange(n, device=DEV)
    slots = table[0].long()[t // page] * page + t % page
    scale = torch.full((3,), 64.0, device=DEV)
    qar.kv_write(k, v, slots, kc, vc, scale)
    assert torch.equal(kc[pages - 1], codes_of(k[:256], 64.0))
    assert torch.equal(vc[7, :44], codes_of(v[256:], 64.0))
    q = torch.randn(1, heads, 128, device=DEV).to(torch.bfloat16)
    seq, cu = dev32([n]), dev32([0, 1])
    out = qar.kv_tree_fwd(q, kc, vc, table, seq, cu, 1, n, 1.0 / scale)
    small = [torch.cat([c[pages - 1], c[7]]).view(2, page, heads, 128) for c in (kc, vc)]
    same = qar.kv_tree_fwd(q, *small, dev32([[0, 1]]), seq, cu, 1, n, 1.0 / scale)
    assert torch.equal(out, same)


# ---------------------------------------------------------------------------
# accepted paths
# ---------------------------------------------------------------------------

def keep_case(seed, rows, page, heads, fp8, layout, deepest):
    r = np.random.Generator(np.random.PCG64(seed))
    g = torch.Generator().manual_seed(seed)
    nodes = r.integers(0, 65, rows)
    nodes[0] = max(1, nodes[0])
    seq = nodes + r.integers(0, 100, rows)
    need = -(-seq // page)
    num = int(need.sum()) + 1
    tables = np.full((rows, max(1, int(need.max()))), -1, dtype=np.int32)
    perm, at = r.permutation(num), 0
    for b in range(rows):
        tables[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    keep = np.minimum(r.integers(0, deepest + 1, rows), nodes)
    paths = np.full((rows, deepest), -1, dtype=np.int32)
    for b in range(rows):
        paths[b, :keep[b]] = np.sort(r.choice(nodes[b], keep[b], replace=False)) if keep[b] else []
    dtype = torch.uint8 if fp8 else torch.bfloat16
    base, kc, vc = cache_views(num, page, heads, dtype, layout)
    rnd = torch.randint(0, 256, (base.numel() * base.element_size(),), generator=g,
                        dtype=torch.uint8)
    base.view(torch.uint8).view(-1).copy_(rnd)
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    return base, kc, vc, tables, seq, cu, paths, keep


def bits(x):
    return x.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("rows,page,heads,fp8,layout,deepest", [
    (1, 16, 1, True, "token", 3), (9, 8, 5, False, "head", 12), (33, 32, 8, True, "interleaved", 64),
    (5, 1024, 16, False, "token", 20), (4, 64, 40, True, "head", 9),
])
def test_keep_path(rows, page, heads, fp8, layout, deepest):
    base, kc, vc, tables, seq, cu, paths, keep = keep_case(rows, rows, page, heads, fp8, layout,
                                                           deepest)
    want = [ref.keep_path(bits(c).reshape(*c.shape[:3], -1), tables, seq, cu, paths, keep)
            for c in (kc, vc)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qar.kv_keep_path(kc, vc, dev32(tables), dev32(seq), dev32(cu), dev32(paths), dev32(keep),
                     error=err)
    torch.cuda.synchronize()
    assert qar.read_error_word(err) == 0
    for c, w in zip((kc, vc), want):
        assert np.array_equal(bits(c).reshape(w.shape), w)


@pytest.mark.parametrize("why,path,keep", [
    ("falls", [3, 2], 2), ("stands", [1, 1], 2), ("leaves the nodes", [0, 6], 2),
    ("starts below 0", [-1, 2], 2), ("longer than the nodes", [0, 1, 2, 3, 4, 5, 6], 7),
    ("negative length", [0, 1], -1), ("beyond the depth", [0, 1], 8),
])
def test_keep_path_leaves_a_request_with_a_bad_path_out(why, path, keep):
    kc = torch.arange(2 * 16, device=DEV).view(2, 16, 1, 1).expand(2, 16, 1, 128).to(torch.bfloat16)
    kc = kc.contiguous()
    vc = kc.clone()
    paths = np.zeros((2, 7), dtype=np.int32)
    paths[0, :len(path)] = path
    paths[1, :2] = [2, 4]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qar.kv_keep_path(kc, vc, dev32([[0], [1]]), dev32([10, 10]), dev32([0, 6, 12]), dev32(paths),
                     dev32([keep, 2]), error=err)
    torch.cuda.synchronize()
    assert qar.read_error_word(err) == 6
    want = list(range(32))
    want[16 + 4], want[16 + 5] = 16 + 6, 16 + 8       # request 1: nodes 2 and 4 -> 0 and 1
    assert kc[:, :, 0, 0].flatten().tolist() == want
    assert torch.equal(kc, vc)


def test_keep_path_page_outside_the_cache():
    kc = torch.randn(2, 16, 1, 128, device=DEV).to(torch.bfloat16)
    vc = torch.randn(2, 16, 1, 128, device=DEV).to(torch.bfloat16)
    before = kc.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    # nodes 0..19 at positions 12..31; the second page is bad, so nodes from 4 on do not move
    qar.kv_keep_path(kc, vc, dev32([[1, 2]]), dev32([32]), dev32([0, 20]), dev32([[1, 3, 7]]),
                     dev32([3]), error=err)
    torch.cuda.synchronize()
    assert qar.read_error_word(err) == 7
    want = before.clone()
    want[1, 12], want[1, 13] = before[1, 13], before[1, 15]
    assert torch.equal(kc, want)
