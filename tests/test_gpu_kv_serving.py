"""GPU: the paged cache operators as a server uses them together -- prompts
admitted, single tokens decoded, trees drafted, verified and rolled back,
requests ended -- for an E4M3 layer with static scales and a layer kept in
bf16, against a plain state of token rows and 64-bit attention."""
import numpy as np
import pytest
import torch

import quantization_amax_reduce_b200 as qar
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
HQ, HKV, PAGE, PAGES, WIDTH, ROWS = 6, 2, 16, 60, 24, 4
BOUNDS = (7.5, 7.0, 7.25)


class Server:
    """Two layers over one pool; `mirror[layer][b]` holds the K and V rows that
    request b's cache must stand for."""

    def __init__(self):
        self.ctx = qar.Context(2)
        self.ctx.set_static_scales(0, *BOUNDS)
        self.skip = np.array([0, 1], dtype=np.uint8)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.tables = torch.full((ROWS, WIDTH), -1, **i32)
        self.owned = torch.zeros(ROWS, **i32)
        self.free = torch.randperm(PAGES, generator=torch.Generator().manual_seed(1)).to(**i32)
        self.pool = torch.tensor([PAGES, 0], **i32)
        self.err = torch.zeros(1, **i32)
        self.caches = []
        for layer in range(2):
            dtype = torch.bfloat16 if self.mode(layer) == qar.SKIP else torch.uint8
            self.caches.append([torch.full((PAGES, PAGE, HKV, 128), 0x7F, dtype=torch.uint8,
                                           device=DEV) if dtype == torch.uint8 else
                                torch.full((PAGES, HKV, PAGE, 128), float("nan"), dtype=dtype,
                                           device=DEV).transpose(1, 2) for _ in range(2)])
        self.seq = np.zeros(ROWS, dtype=np.int64)
        self.mirror = [[np.zeros((0, 2, HKV, 128)) for _ in range(ROWS)] for _ in range(2)]

    def mode(self, layer):
        return self.ctx.select_mode(layer, self.skip)

    def scales(self, layer):
        if self.mode(layer) == qar.SKIP:
            return None, None, (1.0, 1.0, 1.0)
        ds = [float(np.float32(b) / np.float32(448)) for b in BOUNDS]
        return self.ctx.static_quant_scale_ptr(layer), self.ctx.static_descale_ptr(layer), ds

    def step(self, gen, new, pad=0, masks=None):
        """New tokens (a prompt's chunk, a token, or a tree) of every request."""
        new = np.asarray(new)
        total = int(new.sum())
        self.seq = self.seq + new
        seq = torch.as_tensor(self.seq.astype(np.int32), device=DEV)
        cu, slots, positions = qar.kv_assign_pages(
            seq, torch.as_tensor(new.astype(np.int32), device=DEV), self.tables, self.owned,
            self.free, self.pool, PAGE, total + pad, error=self.err)
        want = np.concatenate([np.arange(s - n, s) for s, n in zip(self.seq, new)])
        assert positions[:total].tolist() == want.tolist()
        mask = None
        if masks is not None:
            mask = np.concatenate([np.asarray(m, dtype=np.uint64) for m in masks] +
                                  [np.zeros(pad, dtype=np.uint64)])[:, None]
        for layer in range(2):
            qkv = torch.randn(total + pad, HQ + 2 * HKV, 128, generator=gen).to(torch.bfloat16)
            q, k, v = qkv.to(DEV).split([HQ, HKV, HKV], dim=1)
            quant, descale, ds = self.scales(layer)
            kc, vc = self.caches[layer]
            qar.kv_write(k, v, slots, kc, vc, quant, error=self.err)
            out = torch.full((total + pad, HQ, 128), 4.0, dtype=torch.bfloat16, device=DEV)
            qar.kv_tree_fwd(q, kc, vc, self.tables, seq, cu, int(new.max()), int(self.seq.max()),
                            descale, None if mask is None else
                            torch.as_tensor(mask.view(np.int64), device=DEV), out=out,
                            error=self.err)
            torch.cuda.synchronize()
            assert qar.read_error_word(self.err) == 0
            assert (out[total:] == 4).all()
            # the plain state: what the cache's type makes of the new rows
            at = 0
            for b in range(ROWS):
                rows = []
                for x, bound in ((k, BOUNDS[1]), (v, BOUNDS[2])):
                    x = x[at:at + new[b]].cpu()
                    if self.mode(layer) != qar.SKIP:
                        scale = np.float32(448) / np.float32(bound)
                        x = (x.float() * float(scale)).clamp(-448, 448).to(torch.float8_e4m3fn)
                    rows.append(x.double().numpy())
                self.mirror[layer][b] = np.concatenate(
                    [self.mirror[layer][b], np.stack(rows, axis=1)])
                at += new[b]
            self.check_attention(layer, q[:total].double().cpu().numpy(), new, mask, ds,
                                 out[:total].double().cpu().numpy())

    def check_attention(self, layer, q, new, mask, ds, got):
        kv = self.mirror[layer]
        longest = max(len(m) for m in kv)
        # the plain rows as one page per request
        cache = np.zeros((ROWS, longest, 2, HKV, 128))
        for b, m in enumerate(kv):
            cache[b, :len(m)] = m
        cu = np.concatenate([[0], np.cumsum(new)])
        want, tol = ref.tree_attention(q, cache[:, :, 0], cache[:, :, 1],
                                       np.arange(ROWS)[:, None], [len(m) for m in kv], cu, mask,
                                       None, ds, self.mode(layer) != qar.SKIP)
        assert (np.abs(got - want) <= tol).all()

    def keep(self, nodes, paths):
        """The trees' accepted paths stay, the rest goes."""
        nodes = np.asarray(nodes)
        depth = max(len(p) for p in paths) + 1
        table = np.full((ROWS, depth), -1, dtype=np.int32)
        for b, p in enumerate(paths):
            table[b, :len(p)] = p
        kept = np.array([len(p) for p in paths])
        cu = torch.as_tensor(np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32), device=DEV)
        seq = torch.as_tensor(self.seq.astype(np.int32), device=DEV)
        for layer in range(2):
            qar.kv_keep_path(*self.caches[layer], self.tables, seq, cu,
                             torch.as_tensor(table, device=DEV),
                             torch.as_tensor(kept.astype(np.int32), device=DEV), error=self.err)
            for b, p in enumerate(paths):
                m = self.mirror[layer][b]
                first = len(m) - nodes[b]
                self.mirror[layer][b] = np.concatenate([m[:first], m[[first + i for i in p]]]) \
                    if len(p) else m[:first]
        self.shrink(self.seq - nodes + kept)

    def shrink(self, seq):
        """Requests become shorter (or end, at 0): their last pages go back."""
        self.seq = np.asarray(seq)
        for layer in range(2):
            for b in range(ROWS):
                self.mirror[layer][b] = self.mirror[layer][b][:self.seq[b]]
        none = torch.zeros(ROWS, dtype=torch.int32, device=DEV)
        qar.kv_assign_pages(torch.as_tensor(self.seq.astype(np.int32), device=DEV), none,
                            self.tables, self.owned, self.free, self.pool, PAGE, 0,
                            error=self.err)
        torch.cuda.synchronize()
        assert qar.read_error_word(self.err) == 0
        used = int((-(-self.seq // PAGE)).sum())
        assert self.pool.tolist() == [PAGES - used, 0]


def draft(r, nodes):
    """Ancestor masks of a random tree."""
    words = []
    for i in range(nodes):
        up = words[int(r.integers(0, i))] if i else 0
        words.append(up | 1 << i)
    return words


def test_serving_loop():
    gen = torch.Generator().manual_seed(7)
    r = np.random.Generator(np.random.PCG64(7))
    s = Server()
    s.step(gen, [70, 5, 33, 1], pad=3)             # prompts, in a padded buffer
    s.step(gen, [1, 1, 1, 1])                      # a token each
    s.step(gen, [0, 40, 0, 1])                     # a chunk beside a token
    for nodes in ([7, 1, 12, 5], [20, 3, 1, 9]):   # drafted trees and their verification
        masks = [draft(r, n) for n in nodes]
        s.step(gen, nodes, masks=masks)
        paths = []
        for m in masks:                            # a random leaf's ancestors, cut anywhere
            path = [i for i in range(len(m)) if m[int(r.integers(0, len(m)))] >> i & 1]
            paths.append(path[:int(r.integers(0, len(path) + 1))])
        s.keep(nodes, paths)
        s.step(gen, [1, 1, 1, 1])                  # the next tokens see the kept rows
    s.shrink([0, s.seq[1], 0, s.seq[3]])           # two requests end
    s.step(gen, [100, 1, 0, 1])                    # and another takes a row
    # a step that the pool cannot hold changes nothing, and the server goes on
    before = s.tables.clone()
    seq = torch.as_tensor((s.seq + [0, 300, 300, 300]).astype(np.int32), device=DEV)
    qar.kv_assign_pages(seq, torch.zeros_like(seq), s.tables, s.owned, s.free, s.pool, PAGE, 0,
                        error=s.err)
    torch.cuda.synchronize()
    assert qar.read_error_word(s.err) == 7 and torch.equal(before, s.tables)
    s.step(gen, [1, 1, 17, 1])


def test_static_pointers_follow_the_context():
    ctx = qar.Context(2)
    for get in (ctx.static_quant_scale_ptr, ctx.static_descale_ptr):
        with pytest.raises(qar.FP8AttnError):
            get(0)
    ctx.set_static_scales(1, 224.0, 198.0, 210.0)
    x = torch.full((2, 1, 128), 99.0, dtype=torch.bfloat16, device=DEV)
    cache = [torch.zeros(1, 16, 1, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
    qar.kv_write(x, x, torch.arange(2, device=DEV), *cache, ctx.static_quant_scale_ptr(1))
    # 99 * 448 / 198 = 224 and 99 * 448 / 210 = 211.2 -> 208
    value = lambda c: c.view(torch.float8_e4m3fn).float()[0, :2]      # noqa: E731
    assert (value(cache[0]) == 224).all() and (value(cache[1]) == 208).all()
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)   # noqa: E731
    out = qar.kv_tree_fwd(q, *cache, i32(0).view(1, 1), i32(2), i32(0, 1), 1, 2,
                          ctx.static_descale_ptr(1))
    assert (out == 208 * 210 / 448).all()
    ctx.clear_static_scales(1)
    with pytest.raises(qar.FP8AttnError):
        ctx.static_descale_ptr(1)


def test_argument_checks_launch_nothing():
    i32 = dict(dtype=torch.int32, device=DEV)
    seq, new, owned = (torch.zeros(3, **i32) for _ in range(3))
    tables, free, pool = torch.zeros(3, 4, **i32), torch.zeros(9, **i32), torch.zeros(2, **i32)
    good = [seq, new, tables, owned, free, pool, 16, 8]
    n0 = qar.launch_count()

    def refuse(f, args, match, at=None, value=None, **kw):
        args = list(args)
        if at is not None:
            args[at] = value
        with pytest.raises((ValueError, qar.FP8AttnError), match=match):
            f(*args, **kw)

    f = qar.kv_assign_pages
    refuse(f, good, "CUDA", 0, seq.cpu())
    refuse(f, good, "new_lens", 1, new[:2])
    refuse(f, good, "new_lens", 1, new.long())
    refuse(f, good, "block_tables", 2, tables[:2])
    refuse(f, good, "block_tables", 2, tables[:, :0])
    refuse(f, good, "rows", 2, torch.zeros(4, 3, **i32).t())
    refuse(f, good, "owned", 3, owned[::2])
    refuse(f, good, "free_pages", 4, free.cpu())
    refuse(f, good, "pool", 5, pool[:1])
    refuse(f, good, "unsupported", 6, 20)
    refuse(f, good, "negative", 7, -1)
    refuse(f, good, "needed", out=(torch.zeros(4, **i32), torch.zeros(7, dtype=torch.int64, device=DEV),
                                   torch.zeros(8, **i32)))
    x = torch.zeros(5, 2, 128, dtype=torch.bfloat16, device=DEV)
    slots = torch.arange(5, device=DEV)
    c = [torch.zeros(2, 16, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    c8 = [torch.zeros(2, 16, 2, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scale = torch.ones(3, device=DEV)
    f, good = qar.kv_write, [x, x, slots, *c]
    refuse(f, good, "share", 1, x[:4])
    refuse(f, good, "slots", 2, slots[:4])
    refuse(f, good, "slots", 2, slots.int())
    refuse(f, good + [scale], "takes no")
    refuse(f, [x, x, slots, *c8], "needed")
    refuse(f, [x, x, slots, *c8, scale.double()], "fp32")
    refuse(f, [x, x, slots, c[0], c8[0]], "both be")
    refuse(f, [x[:, :1], x[:, :1], slots, *c], "contiguous channels")
    refuse(f, [x, x, slots, *[t[..., 0:128:1].transpose(0, 3) for t in c]], "cache")
    paths, keep, cu = torch.zeros(3, 2, **i32), torch.zeros(3, **i32), torch.zeros(4, **i32)
    f, good = qar.kv_keep_path, [*c, tables, seq, cu, paths, keep]
    refuse(f, good, "cu_q", 4, cu[:3])
    refuse(f, good, "paths", 5, paths[:2])
    refuse(f, good, "paths", 5, paths.long())
    refuse(f, good, "keep_lens", 6, keep[:2])
    assert qar.launch_count() == n0
    # empty calls launch nothing either
    qar.kv_write(x[:0], x[:0], slots[:0], *c)
    qar.kv_keep_path(*c, tables, seq, cu, paths[:, :0], keep)
    e = torch.zeros(0, **i32)
    cu, _, _ = qar.kv_assign_pages(e, e, tables[:0], e, free, pool, 16, 0)
    assert qar.launch_count() == n0 and cu.tolist() == [0]
