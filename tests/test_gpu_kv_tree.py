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
])
def test_against_64_bits(seq, nodes, hq, hkv, page, fp8):
    s = make(hash((tuple(seq), hq)) % 1000, seq, nodes, hq, hkv, page, fp8, head_major=page > 32)
    check(run(s), *expect(s))
