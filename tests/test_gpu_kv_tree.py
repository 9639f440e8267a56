"""GPU: attention of drafted trees, chains and single tokens over a paged KV
cache (fp8attn_kv_tree_fwd) against a plain 64-bit statement, within the
error that its roundings allow (tests/kv_reference.py)."""
import numpy as np
import pytest
import torch

import quantization_amax_reduce_b200 as qar
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BOUNDS = (7.5, 7.0, 7.25)
NAN_CODE = 0x7F


def make(seed, seq, nodes, hq, hkv, page, fp8, head_major=False, tree=True, spread=1.0, extra=3):
    """A cache of random pages, queries and masks for these requests."""
    g = torch.Generator().manual_seed(seed)
    r = np.random.Generator(np.random.PCG64(seed))
    need = [-(-s // page) for s in seq]
    num = sum(need) + extra
    perm = r.permutation(num).astype(np.int32)
    width = max(1, max(need))
    tables = np.full((len(seq), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = perm[at:at + n]
        at += n
    caches, values = [], []
    for t in (1, 2):
        x = torch.randn(num, page, hkv, 128, generator=g) * spread
        if fp8:
            c = (x * (448.0 / BOUNDS[t])).clamp(-448, 448).to(torch.float8_e4m3fn)
            values.append(c.double().numpy())
            c = c.view(torch.uint8)
        else:
            c = x.to(torch.bfloat16)
            values.append(c.double().numpy())
        c = c.to(DEV)
        if head_major:
            c = c.transpose(1, 2).contiguous().transpose(1, 2)
        caches.append(c)
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    q = (torch.randn(int(cu[-1]), hq, 128, generator=g) * spread).to(torch.bfloat16)
    mask = None
    if tree:
        words = max(1, -(-max(nodes) // 64))
        mask = np.zeros((int(cu[-1]), words), dtype=np.uint64)
        for b, n in enumerate(nodes):
            for i in range(n):
                row = mask[cu[b] + i]
                if i:
                    row |= mask[cu[b] + int(r.integers(0, i))]
                row[i // 64] |= np.uint64(1) << np.uint64(i % 64)
    ds = tuple(np.float32(b / 448.0) for b in BOUNDS) if fp8 else (1.0, 1.0, 1.0)
    return dict(q=q, caches=caches, values=values, tables=tables, seq=np.asarray(seq, np.int32),
                cu=cu, mask=mask, ds=ds, fp8=fp8, max_q=max(nodes), max_seq=max(seq))


def to_dev(s):
    d = lambda x: torch.as_tensor(x, device=DEV)   # noqa: E731
    s["args"] = [s["q"].to(DEV), s["caches"][0], s["caches"][1], d(s["tables"]), d(s["seq"]),
                 d(s["cu"]), s["max_q"], s["max_seq"],
                 d(np.asarray(s["ds"], np.float32)) if s["fp8"] else None,
                 None if s["mask"] is None else d(s["mask"].view(np.int64))]
    return s["args"]


def expect(s, scale=None):
    return ref.tree_attention(s["q"].double().numpy(), s["values"][0], s["values"][1], s["tables"],
                              s["seq"], s["cu"], s["mask"], scale, [float(x) for x in s["ds"]],
                              s["fp8"])


def check(got, want, tol, what=""):
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    worst = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err) - tol), err.shape)
    assert (err <= tol).all(), \
        f"{what}: at {worst} got {got[worst]} want {want[worst]} tolerance {tol[worst]}; " \
        f"{(~(err <= tol)).sum()} of {err.size} outside"


def run(s, **kw):
    args = to_dev(s)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = qar.kv_tree_fwd(*args, error=err, **kw)
    torch.cuda.synchronize()
    assert qar.read_error_word(err) == 0
    return out


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("seq,nodes,hq,hkv,page", [
    ([1], [1], 1, 1, 16),                    # one token, its own key
    ([128], [1], 8, 1, 16),                  # one whole tile
    ([129], [1], 16, 2, 32),                 # one key in the second tile
    ([300], [5], 4, 4, 64),                  # a KV head for every query head
    ([700, 33, 5], [7, 3, 5], 10, 2, 16),    # five query heads to a KV head
    ([257, 1000], [64, 20], 8, 1, 128),      # many row tiles of 64
    ([90], [20], 2, 2, 8),                   # the smallest pages; 32 columns
    ([1500, 40], [2, 30], 32, 8, 256),       # pages larger than a tile
    ([2100], [3], 4, 1, 1024),
    ([300, 1], [9, 1], 4, 1, 16),            # 36 rows: two copies on the lanes
    ([513], [16], 4, 1, 32),                 # 64 rows, one key in the fifth tile
    ([400], [13], 5, 1, 16),                 # 65 rows
    ([640, 129], [16, 17], 8, 1, 64),        # 128 rows; 136: a second tile of 8
    ([5000], [3], 4, 2, 64),                 # cut over many CTAs
    ([3000, 2900], [10, 1], 8, 2, 16),       # the same with 40 rows a KV head
    ([2500], [20], 8, 1, 128),               # and with 160
])
def test_against_64_bits(seq, nodes, hq, hkv, page, fp8):
    s = make(hash((tuple(seq), hq)) % 1000, seq, nodes, hq, hkv, page, fp8, head_major=page > 32)
    check(run(s), *expect(s))


def brute_fill(s, what):
    """Overwrites every slot that no request holds, and the rest of last pages."""
    held = np.zeros(s["values"][0].shape[:2], dtype=bool)
    page = held.shape[1]
    for b, n in enumerate(s["seq"]):
        for p in range(int(n)):
            held[s["tables"][b][p // page], p % page] = True
    at = torch.from_numpy(np.argwhere(~held)).to(DEV)
    for c in s["caches"]:
        c[at[:, 0], at[:, 1]] = what


def set_kv(s, t, b, pos, channel, value):
    """K (t = 0) or V (1) of request b's position, one channel of every head."""
    page = s["values"][t].shape[1]
    where = s["tables"][b][pos // page], pos % page
    if s["fp8"]:
        assert np.isnan(value)
        s["caches"][t][where][:, channel] = NAN_CODE
    else:
        s["caches"][t][where][:, channel] = value
    s["values"][t][where][:, channel] = value


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("nodes,hq,hkv", [(4, 4, 2), (20, 2, 2), (20, 4, 2), (33, 4, 1), (100, 2, 2)])
def test_masks_with_empty_rows_and_several_words(nodes, hq, hkv, fp8):
    s = make(nodes, [nodes, nodes + 200], [nodes, nodes], hq, hkv, 16, fp8)
    s["mask"][2] = 0                       # sees nothing at all
    s["mask"][nodes + 1] = 0               # sees the context alone
    s["mask"][nodes - 1] = np.uint64(1)    # sees the root, not itself
    if nodes > 64:
        s["mask"][nodes - 2] = [0, 1 << 20]       # a node of the second word alone
    # bits past the nodes mean nothing
    s["mask"][0, -1] |= np.uint64(1) << np.uint64(63)
    want, tol = expect(s)
    assert (want[2] == 0).all()
    got = run(s)
    assert (got[2] == 0).all()
    check(got, want, tol)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("nodes,hq,hkv", [(4, 4, 2), (20, 2, 2), (20, 4, 2), (33, 4, 1)])
def test_non_finite_values_in_hidden_places(nodes, hq, hkv, fp8):
    """NaN and Inf in slots of no request, and in nodes that a query does not
    see, do not touch it; a query that sees them shows them."""
    s = make(nodes + 7, [nodes + 130, nodes + 61], [nodes, nodes], hq, hkv, 16, fp8)
    brute_fill(s, NAN_CODE if fp8 else float("nan"))
    first = 130
    bad = float("nan") if fp8 else float("inf")
    set_kv(s, 1, 0, first + 1, 5, bad)               # V of node 1 of request 0
    set_kv(s, 1, 0, first + 2, 9, float("nan"))      # V of node 2
    set_kv(s, 0, 0, first + 3, 17, float("nan"))     # K of node 3
    sees = (s["mask"][:nodes, :1] >> np.arange(min(nodes, 64), dtype=np.uint64)) & 1
    got = run(s).double().cpu().numpy()
    want, tol = expect(s)
    for i in range(nodes):
        if sees[i, 3]:
            assert np.isnan(got[i]).all()
            want[i], got[i] = 0, 0
            continue
        for node, channel in ((1, 5), (2, 9)):
            if sees[i, node]:
                v = got[i, :, channel]
                assert np.isnan(v).all() if node == 2 or fp8 else (v == np.inf).all()
                want[i, :, channel] = got[i, :, channel] = 0
    assert np.isfinite(want).all()
    check(torch.from_numpy(got), want, np.nan_to_num(tol, nan=1.0, posinf=1.0))
    # the other request never met any of it
    check(torch.from_numpy(got[nodes:]), want[nodes:], tol[nodes:])


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("nodes,hq,hkv", [(1, 8, 1), (4, 5, 1), (12, 4, 1), (30, 4, 1)])
def test_references_that_move_and_far_tails(nodes, hq, hkv, fp8):
    """Scores that grow along the sequence move the reference again and again;
    a sink key 2^-17 above thousands of equal ones must not swallow them."""
    L = 1500
    s = make(nodes, [L], [nodes], hq, hkv, 32, fp8, tree=False)
    ramp = np.linspace(0.02, 1.0, L)
    page = 32
    q = s["q"].float()
    q[:] = torch.sign(q) * 2.0
    s["q"] = q.to(torch.bfloat16)
    for p in range(L):
        at = s["tables"][0][p // page], p % page
        k = s["values"][0][at]
        k[:] = np.sign(s["q"][0, 0].double().numpy()) * ramp[p] * (64 if fp8 else 1)
    c = torch.from_numpy(s["values"][0])
    c = c.to(torch.float8_e4m3fn) if fp8 else c.to(torch.bfloat16)
    s["values"][0][:] = c.double().numpy()
    s["caches"][0] = (c.view(torch.uint8) if fp8 else c).to(DEV)
    check(run(s), *expect(s))
    # the sink: one key along q, the others orthogonal to it (zero)
    s["values"][0][:] = 0
    at = s["tables"][0][3 // page], 3 % page
    unit = np.sign(s["q"][0, 0].double().numpy())
    scale = 11.78 * np.sqrt(128) / (256 * float(s["ds"][1]))     # exp(11.78) = 2^17
    c = torch.from_numpy(unit * scale)
    c = c.to(torch.float8_e4m3fn) if fp8 else c.to(torch.bfloat16)
    s["values"][0][at] = c.double().numpy()
    s["caches"][0].zero_()
    s["caches"][0][at] = (c.view(torch.uint8) if fp8 else c).to(DEV)
    check(run(s), *expect(s))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("nodes,hq,hkv", [(2, 8, 1), (7, 4, 1), (13, 4, 1), (30, 4, 1), (40, 4, 1)])
def test_references_that_move_inside_a_tile(nodes, hq, hkv, fp8):
    """Scores that climb (for every other query: fall) by 2^9 and 2^18 every 32
    keys, within each tile and a little higher in each, over several tiles."""
    L, page = 900, 16
    s = make(40 + nodes, [L], [nodes], hq, hkv, page, fp8)
    unit = np.sign(s["q"][0, 0].double().numpy())
    rows = np.arange(nodes * hq).reshape(nodes, hq)
    size = np.where(rows % 2, -4.0, 4.0) / (1 + rows // 2 % 2)
    s["q"] = torch.from_numpy(size[..., None] * unit).to(torch.bfloat16)
    for p in range(L):
        level = (0.02 + 0.14 * (p // 16 % 8)) * (0.3 + 0.7 * p / L)
        s["values"][0][s["tables"][0][p // page], p % page] = unit * level * (64 if fp8 else 1)
    c = torch.from_numpy(s["values"][0])
    c = c.to(torch.float8_e4m3fn) if fp8 else c.to(torch.bfloat16)
    s["values"][0][:] = c.double().numpy()
    s["caches"][0] = (c.view(torch.uint8) if fp8 else c).to(DEV)
    check(run(s), *expect(s))


@pytest.mark.parametrize("nodes,hq,hkv", [(6, 2, 1), (6, 4, 1), (12, 4, 1), (40, 4, 1)])
def test_query_rows_of_very_different_sizes(nodes, hq, hkv):
    """E4M3: rows that cannot share a scale, rows of zeros, one with an infinity."""
    s = make(5, [200], [nodes], hq, hkv, 16, True, tree=False)
    size = torch.tensor([2.0 ** ((i * 7) % 23 - 11) for i in range(nodes)])
    s["q"] = (s["q"].float() * size[:, None, None]).to(torch.bfloat16)
    s["q"][3] = 0
    want, tol = expect(s)
    check(run(s), want, tol)
    s["q"][2, 0, 77] = float("inf")
    got = run(s)
    assert torch.isnan(got[2, 0]).all()
    got[2, 0] = 0
    want[2, 0] = 0
    check(got, want, tol)


@pytest.mark.parametrize("fp8", [True, False])
def test_many_requests_some_without_queries(fp8):
    r = np.random.Generator(np.random.PCG64(1))
    B = 1100
    nodes = [int(x) for x in r.integers(0, 4, B)]
    seq = [n + int(x) for n, x in zip(nodes, r.integers(0, 40, B))]
    seq[17] = 700
    s = make(3, seq, nodes, 2, 1, 16, fp8, tree=False)
    check(run(s), *expect(s))


def test_strided_queries_a_scale_and_rows_of_no_request():
    s = make(9, [300, 20], [5, 3], 8, 2, 64, True)
    args = to_dev(s)
    T = s["q"].shape[0]
    wide = torch.zeros(T + 4, 3, 8, 128, dtype=torch.bfloat16, device=DEV)
    wide[:T, 1] = args[0]
    wide[T:, 1] = 7
    out = torch.full((T + 4, 8, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    mask = torch.cat([args[9], args[9][:4]])
    got = qar.kv_tree_fwd(wide[:, 1], *args[1:9], mask, 0.03, out=out)
    assert got is out and (out[T:] == 5).all()
    check(out[:T], *expect(s, np.float64(np.float32(0.03))))


def test_bad_requests_are_left_out_and_reported():
    s = make(4, [40, 50, 60, 70], [4, 5, 6, 7], 4, 2, 16, True, tree=False)
    want, tol = expect(s)
    args = to_dev(s)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def attempt(**change):
        a = list(args)
        for i, v in change.items():
            a[int(i[1:])] = v
        out = torch.full(args[0].shape, 9.0, dtype=torch.bfloat16, device=DEV)
        qar.kv_tree_fwd(*a, out=out, error=err)
        torch.cuda.synchronize()
        return out, qar.read_error_word(err)

    seq = args[4].clone()
    seq[1] = 4                                    # shorter than its five queries
    seq[2] = 16 * args[3].shape[1] + 1            # beyond the block table
    out, status = attempt(a4=seq, a7=4000)
    assert status == 6 and (out[4:15] == 9).all()
    check(out[:4], want[:4], tol[:4])
    check(out[15:], want[15:], tol[15:])
    out, status = attempt(a6=6)                   # the last request has seven
    assert status == 6 and (out[15:] == 9).all()
    check(out[:15], want[:15], tol[:15])
    out, status = attempt(a7=60)                  # and is longer than 60
    assert status == 6 and (out[15:] == 9).all()
    cu = args[5].clone()
    cu[4] = 23                                    # beyond the queries
    out, status = attempt(a5=cu)
    assert status == 6 and (out[15:] == 9).all()
    # a page id outside the cache reads as zeros
    tables = args[3].clone()
    tables[3, 1], tables[0, 2] = 10 ** 6, -3
    out, status = attempt(a3=tables)
    assert status == 7
    zero = len(s["values"][0])
    s["values"] = [np.concatenate([v, np.zeros_like(v[:1])]) for v in s["values"]]
    s["tables"][3, 1], s["tables"][0, 2] = zero, zero
    check(out, *expect(s))


def test_argument_checks_launch_nothing():
    s = make(2, [40], [4], 4, 2, 16, True)
    a = to_dev(s)
    n0 = qar.launch_count()

    def refuse(match, **change):
        b = list(a)
        kw = {}
        for k, v in change.items():
            if k[0] == "a" and k[1:].isdigit():
                b[int(k[1:])] = v
            else:
                kw[k] = v
        with pytest.raises((ValueError, qar.FP8AttnError), match=match):
            qar.kv_tree_fwd(*b, **kw)

    refuse("CUDA", a0=a[0].cpu())
    refuse("bfloat16", a0=a[0].float())
    refuse("heads", a0=a[0][:, :3])
    refuse("128", a0=a[0][..., :64])
    refuse("both be", a1=a[1].view(torch.int8), a2=a[2].view(torch.int8))
    refuse("share", a2=a[2][:2])
    refuse("block_tables", a3=a[3].long())
    refuse("block_tables", a3=a[3][:, 0])
    refuse("seq_lens", a4=a[4].long())
    refuse("cu_q", a5=a[5][:1])
    refuse("needed", a8=None)
    refuse("tree_mask", a9=a[9][:2])
    refuse("tree_mask", a9=a[9].int())
    refuse("invalid", softmax_scale=-1.0)
    refuse("invalid", softmax_scale=float("nan"))
    refuse("needed", out=torch.zeros(3, 4, 128, dtype=torch.bfloat16, device=DEV))
    refuse("int32", error=torch.zeros(1, device=DEV))
    bf = [x.view(torch.bfloat16)[..., :64].contiguous() for x in a[1:3]]
    refuse("128", a1=bf[0], a2=bf[1])
    odd = torch.zeros(4, 24, 2, 128, dtype=torch.uint8, device=DEV)
    refuse("unsupported", a1=odd, a2=odd)
    assert qar.launch_count() == n0


def test_same_bits_again_on_another_stream_and_replayed():
    """Results do not depend on timing: calls repeated, overlapping on two
    streams, captured and replayed with other lengths give the same bits."""
    s = make(8, [6000, 400, 1, 77], [7, 1, 1, 4], 16, 2, 64, True, tree=False)
    big = make(9, [3000, 900], [30, 20], 16, 2, 64, True)
    args, more = to_dev(s), to_dev(big)
    one, two = qar.kv_tree_fwd(*args), qar.kv_tree_fwd(*more)
    assert torch.equal(one, qar.kv_tree_fwd(*args))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(10):
        outs.append((qar.kv_tree_fwd(*args, stream=streams[0]),
                     qar.kv_tree_fwd(*more, stream=streams[1])))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, one) and torch.equal(b, two)
    raw = qar.kv_tree_fwd(*args, stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(raw, one)
    # two graphs over the same inputs and outputs, replayed with other lengths
    args[7] = 6400
    out = torch.empty_like(one)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qar.kv_tree_fwd(*args, out=out)
        graphs.append(g)
    for lens in ([6000, 400, 1, 77], [130, 390, 1, 4], [7, 1, 1, 64]):
        args[4].copy_(torch.tensor(lens, dtype=torch.int32))
        want = qar.kv_tree_fwd(*args)
        for g in graphs:
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("nodes,hq,hkv,length", [(48, 32, 8, 4100), (32, 32, 8, 4100),
                                                 (4, 64, 8, 4100), (1, 16, 2, 9000),
                                                 (3, 16, 16, 152)])
def test_same_bits_over_many_runs(nodes, hq, hkv, length, fp8):
    """Results do not depend on timing: a hundred runs, with the rings of tiles
    full, against the first."""
    args = to_dev(make(31, [length] * 8, [nodes] * 8, hq, hkv, 64, fp8, head_major=True))
    first = qar.kv_tree_fwd(*args)
    differ = sum((qar.kv_tree_fwd(*args) != first).any().long() for _ in range(100))
    assert int(differ) == 0



@pytest.mark.parametrize("fp8", [True, False])
def test_requests_that_share_pages(fp8):
    """A common prompt lies in the cache once; one request appears twice."""
    s = make(33, [300, 300, 300, 260], [9, 9, 9, 1], 8, 2, 16, fp8)
    s["tables"][1, :17] = s["tables"][0, :17]      # 272 of the 291 tokens of context
    s["tables"][2] = s["tables"][0]
    s["tables"][3, :16] = s["tables"][0, :16]
    check(run(s), *expect(s))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("nodes", [1, 2])
def test_a_thousand_query_heads_to_a_kv_head(nodes, fp8):
    s = make(34, [400, nodes], [nodes, nodes], 1024, 1, 32, fp8)
    check(run(s), *expect(s))


@pytest.mark.parametrize("fp8", [True, False])
def test_mask_bits_beyond_the_nodes_are_ignored(fp8):
    s = make(35, [200, 90, 64], [5, 64, 33], 4, 2, 16, fp8)
    want = run(s)
    for b in range(3):
        n = int(s["cu"][b + 1] - s["cu"][b])
        if n < 64:
            s["mask"][s["cu"][b]:s["cu"][b + 1], 0] |= np.uint64((1 << 64) - (1 << n))
    assert torch.equal(run(s), want)


def test_two_graphs_replayed_side_by_side():
    """Each graph has its own workspace, whatever the other one does meanwhile."""
    sets = [to_dev(make(36, [5000, 700, 3000], [2, 2, 1], 16, 2, 64, True)),
            to_dev(make(37, [4000, 2500], [40, 64], 16, 4, 16, False))]
    want = [qar.kv_tree_fwd(*a) for a in sets]
    outs = [torch.empty_like(w) for w in want]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for a, out in zip(sets, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                qar.kv_tree_fwd(*a, out=out)
        graphs.append(g)
    for _ in range(20):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out, w)



def test_empty_calls():
    s = make(2, [40], [4], 4, 2, 16, False)
    a = to_dev(s)
    n0 = qar.launch_count()
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    out = qar.kv_tree_fwd(a[0][:0], a[1], a[2], a[3][:0], none, torch.zeros(1, dtype=torch.int32,
                                                                         device=DEV), 0, 0)
    assert out.shape == (0, 4, 128) and qar.launch_count() == n0
    # requests without queries, and no keys at all
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    out = torch.full((1, 4, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qar.kv_tree_fwd(a[0][:1], a[1], a[2], a[3], zero[:1], zero, 0, 0, out=out, error=err)
    torch.cuda.synchronize()
    assert (out == 3).all() and qar.read_error_word(err) == 0


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("nodes", [1, 7, 20])       # 16 and 32 columns, rows on the lanes
@pytest.mark.parametrize("bad", [-2, -1, -(2 ** 31), "end", 2 ** 31 - 1])
def test_any_page_id_outside_the_cache_reads_as_zeros(bad, nodes, fp8):
    """Whatever the id is, its page's keys and values are zeros, not what an
    earlier tile left in shared memory, and the call reports it."""
    s = make(41, [300, 150, 300], [nodes] * 3, 4, 1, 16, fp8)
    run(s)                                            # (shared memory is full of rows now)
    zero = len(s["values"][0])
    args = to_dev(s)
    tables = args[3].clone()
    for b, page in ((0, 12), (1, 0), (2, 18)):        # the last: the page of the nodes
        tables[b, page] = zero if bad == "end" else bad
        s["tables"][b, page] = zero
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = qar.kv_tree_fwd(*args[:3], tables, *args[4:], error=err)
    torch.cuda.synchronize()
    assert qar.read_error_word(err) == 7
    s["values"] = [np.concatenate([v, np.zeros_like(v[:1])]) for v in s["values"]]
    check(out, *expect(s))


@pytest.mark.parametrize("which,tile", [("k", 0), ("v", 0), ("k", 11), ("v", 14)])
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("nodes", [1, 4, 20])       # 16 and 32 columns, rows on the lanes
def test_waits_that_give_up_end_the_call_with_a_timeout(nodes, fp8, which, tile):
    """Loads that never come, at the start of a CTA's range or behind several of
    its units: every wait ends, the call reports it, and the next one is right."""
    seq = [1500, 200, 77, 900] * 12                 # some 26 tiles and their units a CTA
    args = to_dev(make(43, seq, [nodes] * 48, 40, 8, 64, fp8))
    want = qar.kv_tree_fwd(*args)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qar.selftest_kv_tree_stall(which, tile)
    qar.kv_tree_fwd(*args, error=err)
    torch.cuda.synchronize()
    assert qar.read_error_word(err) == 3
    for _ in range(3):
        assert torch.equal(qar.kv_tree_fwd(*args, error=err), want)
    assert qar.read_error_word(err) == 0


def test_a_stall_behind_the_last_tile_changes_nothing():
    args = to_dev(make(44, [700, 30], [3, 1], 8, 2, 16, True))
    want = qar.kv_tree_fwd(*args)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qar.selftest_kv_tree_stall("k", 10 ** 6)
    assert torch.equal(qar.kv_tree_fwd(*args, error=err), want)
    assert qar.read_error_word(err) == 0
