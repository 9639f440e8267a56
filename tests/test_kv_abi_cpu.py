"""The paged KV cache entry points refuse what they cannot compute on the host,
before any CUDA call, and do nothing for empty calls (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED = 0, 1, 4


@pytest.fixture(scope="module")
def L():
    from quantization_amax_reduce_b200 import build
    build.build()
    import quantization_amax_reduce_b200 as qar
    return qar.lib()


def call(fn, base, **change):
    args = dict(base)
    assert set(change) <= set(args)
    args.update(change)
    return fn(*args.values())


def test_assign_pages_refusals(L):
    base = dict(seq=P(16), new=P(16), rows=4, page=16, tables=P(16), stride=8, width=8,
                owned=P(16), free=P(16), num=32, pool=P(16), tokens=64, cu=P(16), slots=P(16),
                pos=P(16), err=None, stream=None)
    f = L.fp8attn_kv_assign_pages
    for change in (dict(rows=-1), dict(num=0), dict(width=0), dict(tokens=-1), dict(page=0),
                   dict(stride=7), dict(seq=None), dict(new=None), dict(tables=None),
                   dict(owned=None), dict(free=None), dict(pool=None), dict(cu=None),
                   dict(slots=None), dict(pos=None), dict(slots=P(8)), dict(pos=P(8)),
                   dict(rows=0)):
        assert call(f, base, **change) == INVALID, change
    for change in (dict(page=4), dict(page=24), dict(page=2048), dict(rows=16385),
                   dict(num=1 << 30), dict(tokens=1 << 31)):
        assert call(f, base, **change) == UNSUPPORTED, change
    assert call(f, base, rows=0, tokens=0) == OK


WRITE = dict(k=P(16), v=P(16), tok=1024, head=128, slots=P(16), tokens=5, heads=8, dim=128,
             kc=P(16), vc=P(16), page_stride=16384, slot_stride=1024, chead=128, num=32, page=16,
             qs=P(16), err=None, stream=None)


def test_write_refusals(L):
    f = L.fp8attn_kv_write
    for change in (dict(tokens=-1), dict(num=0), dict(heads=0), dict(page=0), dict(k=None),
                   dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None)):
        assert call(f, WRITE, **change) == INVALID, change
    for change in (dict(dim=64), dict(page=12), dict(tok=1001), dict(head=0), dict(k=P(8)),
                   dict(kc=P(8)), dict(vc=P(24)), dict(slots=P(4)), dict(page_stride=16392),
                   dict(slot_stride=64), dict(chead=136), dict(page_stride=1 << 38),
                   dict(tokens=1 << 28)):
        assert call(f, WRITE, **change) == UNSUPPORTED, change
    # 8-channel strides are 16 bytes of bf16, but not of E4M3
    assert call(f, WRITE, chead=136, qs=None, tokens=0) == OK
    assert call(f, WRITE, tokens=0, k=None, v=None, slots=None) == OK


TREE = dict(q=P(16), qt=4096, qh=128, kc=P(16), vc=P(16), page_stride=16384, slot_stride=1024,
            chead=128, num=32, page=16, tables=P(16), stride=8, width=8, seq=P(16), cu=P(16),
            rows=3, max_q=4, max_seq=128, total=12, heads=32, kv=8, dim=128, ds=P(16),
            mask=P(16), words=1, scale=0.0, out=P(16), ws=P(16), ws_bytes=1 << 30, err=None,
            stream=None)


def test_tree_refusals(L):
    f = L.fp8attn_kv_tree_fwd
    for change in (dict(rows=-1), dict(max_q=-1), dict(max_seq=-1), dict(total=-1), dict(heads=0),
                   dict(kv=0), dict(heads=30), dict(width=0), dict(words=0), dict(scale=-1.0),
                   dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None),
                   dict(out=None), dict(tables=None), dict(seq=None), dict(cu=None),
                   dict(kc=None), dict(vc=None), dict(num=0), dict(stride=7)):
        assert call(f, TREE, **change) == INVALID, change
    for change in (dict(dim=64), dict(page=48), dict(rows=2049), dict(qt=4100), dict(qh=0),
                   dict(q=P(8)), dict(out=P(8)), dict(mask=P(4)), dict(total=1 << 27),
                   dict(chead=120), dict(ws=P(8))):
        assert call(f, TREE, **change) == UNSUPPORTED, change
    # bounds that allow 2^31 tiles and more
    assert call(f, TREE, rows=2048, kv=32, width=1 << 20, stride=1 << 20,
                max_seq=1 << 24) == UNSUPPORTED
    need = L.fp8attn_kv_tree_workspace_bytes(64, 4, 4096, 32, 8)
    assert need > 0
    big = dict(rows=64, max_seq=4096, width=256, stride=256, total=256)
    assert call(f, TREE, ws_bytes=need - 1, **big) == INVALID
    assert call(f, TREE, ws=None, ws_bytes=need, **big) == INVALID
    assert call(f, TREE, rows=0) == OK
    assert call(f, TREE, total=0, q=None, out=None) == OK


def test_tree_sizes_beyond_32_bits(L):
    f = L.fp8attn_kv_tree_fwd
    # a tile's end would pass 2^31 (pages may repeat in a table)
    long = dict(rows=1, kv=32, page=1024, width=1 << 21, max_seq=(1 << 31) - 1, total=1, max_q=1)
    assert call(f, TREE, **long) == UNSUPPORTED
    assert call(f, TREE, **dict(long, max_seq=(1 << 31) - 256), ws_bytes=0) == INVALID   # (workspace)
    # heads x requests x key tiles: 2^30 x 2^11 x (2^24 - 2) tiles
    assert call(f, TREE, rows=2048, page=1024, width=1 << 21, stride=1 << 21,
                max_seq=(1 << 31) - 256, total=1, max_q=1, heads=1 << 30,
                kv=1 << 30) == UNSUPPORTED
    assert L.fp8attn_kv_tree_workspace_bytes(2048, (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1,
                                             (1 << 31) - 1) > 0
    for change in (dict(heads=2050, kv=2), dict(heads=1024, kv=1, max_q=1 << 20, total=1 << 20)):
        assert call(f, TREE, **change) == UNSUPPORTED, change


def test_tree_workspace(L):
    f = L.fp8attn_kv_tree_workspace_bytes
    for bad in ((0, 1, 1, 1, 1), (1, 0, 1, 1, 1), (1, 1, 0, 1, 1), (1, 1, 1, 3, 2), (1, 1, 1, 0, 1),
                (2049, 1, 1, 1, 1)):
        assert f(*bad) == 0
    # grows with each bound, and stops at a CTA per SM
    assert f(1, 1, 128, 8, 8) <= f(1, 1, 1 << 20, 8, 8) <= f(8, 1, 1 << 20, 8, 8)
    assert f(8, 1, 1 << 20, 8, 8) <= f(8, 64, 1 << 20, 8, 8) <= 2 * 148 * 128 * (128 * 4 + 8) + 148 * 20


def test_keep_path_refusals(L):
    base = dict(kc=P(16), vc=P(16), page_stride=16384, slot_stride=1024, chead=128, num=32,
                page=16, elem=1, heads=8, dim=128, tables=P(16), stride=8, width=8, seq=P(16),
                cu=P(16), rows=3, paths=P(16), path_stride=5, depth=5, keep=P(16), err=None,
                stream=None)
    f = L.fp8attn_kv_keep_path
    for change in (dict(rows=-1), dict(depth=-1), dict(elem=4), dict(width=0), dict(tables=None),
                   dict(seq=None), dict(cu=None), dict(paths=None), dict(keep=None),
                   dict(path_stride=4), dict(stride=7), dict(kc=None), dict(num=0)):
        assert call(f, base, **change) == INVALID, change
    for change in (dict(dim=96), dict(page=7), dict(kc=P(8)), dict(slot_stride=1000)):
        assert call(f, base, **change) == UNSUPPORTED, change
    assert call(f, base, rows=0) == OK
    assert call(f, base, depth=0) == OK


def test_keep_path_heads_beyond_the_grid(L):
    heads = 1 << 18   # 32 bf16 vectors a head, 128 a block: 65536 blocks, one too many
    args = (P(16), P(16), 8 * 128 * heads, 128 * heads, 128, 32, 8, 2, heads, 128, P(16), 8, 8,
            P(16), P(16), 3, P(16), 5, 5, P(16), None, None)
    assert L.fp8attn_kv_keep_path(*args) == UNSUPPORTED


def test_static_pointers_need_a_context(L):
    assert L.fp8attn_static_quant_scale_ptr(None, 0) is None
    assert L.fp8attn_static_descale_ptr(None, 0) is None
    assert L.fp8attn_status_string(7) == b"page outside the cache, or too few free pages"


def test_python_refuses_host_tensors():
    import quantization_amax_reduce_b200 as qar
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(2, 16, 1, 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        qar.kv_assign_pages(i, i, torch.zeros(2, 4, dtype=torch.int32), i, i, i, 16, 0)
    with pytest.raises(ValueError, match="CUDA"):
        qar.kv_write(c, c, i, c, c)
    with pytest.raises(ValueError, match="CUDA"):
        qar.kv_tree_fwd(c, c, c, i, i, i, 1, 1)
    with pytest.raises(ValueError, match="CUDA"):
        qar.kv_keep_path(c, c, i, i, i, i, i)


def test_native_calls_pass_their_arguments_on(L):
    """The CPython calls give the entry points' own answers, argument for
    argument, and refuse what these would not see."""
    import quantization_amax_reduce_b200 as qar
    C = qar._native()
    plain = lambda d: [x.value or 0 if isinstance(x, P) else 0 if x is None else x  # noqa: E731
                       for x in d.values()]
    assert C.write(*plain(dict(WRITE, tokens=0))) == OK
    assert C.tree_fwd(*plain(dict(TREE, rows=0))) == OK
    for k, v, status in (("dim", 64, UNSUPPORTED), ("page", 12, UNSUPPORTED), ("num", 0, INVALID),
                         ("heads", 0, INVALID), ("slot_stride", 64, UNSUPPORTED), ("k", P(8), UNSUPPORTED),
                         ("slots", None, INVALID), ("chead", 136, UNSUPPORTED)):
        assert C.write(*plain(dict(WRITE, **{k: v}))) == status, k
    for k, v, status in (("scale", float("nan"), INVALID), ("words", 0, INVALID), ("qt", 4100, UNSUPPORTED),
                         ("width", 0, INVALID), ("rows", 2049, UNSUPPORTED), ("ws", P(8), UNSUPPORTED),
                         ("out", P(8), UNSUPPORTED), ("kv", 0, INVALID), ("stride", 7, INVALID)):
        assert C.tree_fwd(*plain(dict(TREE, **{k: v}))) == status, k
    for call, good in ((C.write, WRITE), (C.tree_fwd, TREE)):
        with pytest.raises(TypeError, match="number of arguments"):
            call(*plain(good)[:-1])
        with pytest.raises(TypeError, match="number of arguments"):
            call(*plain(good), 0)
        with pytest.raises(ValueError, match="fit an int"):
            call(*plain(dict(good, num=1 << 40)))
        with pytest.raises(TypeError):
            call(*plain(dict(good, num="16")))
    with pytest.raises(ValueError, match="x must be an int32 tensor on cuda:0"):
        C.int32_ptr([1], "x", 0, -1)
    t = torch.zeros(4, 6, dtype=torch.int32)   # (a host tensor is on device -1)
    with pytest.raises(ValueError, match="x must be an int32 tensor on cuda:0"):
        C.int32_ptr(t, "x", 0, -1)
    with pytest.raises(ValueError, match="int32"):
        C.int32_ptr(t.long(), "x", -1, -1)
    with pytest.raises(ValueError, match="x must be contiguous and hold 5 elements"):
        C.int32_ptr(t, "x", -1, 5)
    with pytest.raises(ValueError, match="x must be contiguous$"):
        C.int32_ptr(t.t(), "x", -1, -1)
    assert C.int32_ptr(t[2:], "x", -1, 12) == t.data_ptr() + 48


def test_reference_pool_restores_its_list():
    """The definition's own property: taking pages and giving the same ones
    back leaves the free list as it was (mixed growth and shrinkage between)."""
    from tests.kv_reference import Pool
    r = np.random.Generator(np.random.PCG64(4))
    p = Pool(6, 20, 90, 16, r.permutation(90))
    lens = r.integers(0, 100, 6)
    assert p.assign(lens, lens, 600) is not None
    before, owned = list(p.free), list(p.owned)
    more = lens + r.integers(0, 60, 6)
    assert p.assign(more, more - lens, 600) is not None
    assert p.assign(lens, lens * 0, 0) is not None
    assert p.free == before and p.owned == owned
    assert p.assign(lens + 400, lens * 0, 0) is None and p.free == before


def test_a_missing_scale_does_not_make_a_bf16_cache(L):
    """The scale getters give NULL for a layer without static scales.  Passed
    on, it must not be read as "bf16": twice the cache's bytes would be written
    or read.  A bf16 cache has entry points of its own."""
    assert call(L.fp8attn_kv_write, WRITE, qs=None) == INVALID
    assert call(L.fp8attn_kv_tree_fwd, TREE, ds=None) == INVALID
    write, tree = dict(WRITE), dict(TREE)
    del write["qs"], tree["ds"]
    f = L.fp8attn_kv_write_bf16
    assert call(f, write, tokens=0) == OK
    assert call(f, write, chead=136, tokens=0) == OK      # 16 bytes of bf16
    for change, status in ((dict(tokens=-1), INVALID), (dict(k=None), INVALID),
                           (dict(vc=None), INVALID), (dict(num=0), INVALID),
                           (dict(dim=64), UNSUPPORTED), (dict(chead=132), UNSUPPORTED),
                           (dict(kc=P(8)), UNSUPPORTED), (dict(tok=1001), UNSUPPORTED),
                           (dict(tokens=1 << 28), UNSUPPORTED)):
        assert call(f, write, **change) == status, change
    f = L.fp8attn_kv_tree_fwd_bf16
    assert call(f, tree, rows=0) == OK
    assert call(f, tree, total=0, q=None, out=None) == OK
    for change, status in ((dict(max_q=-1), INVALID), (dict(scale=-1.0), INVALID),
                           (dict(words=0), INVALID), (dict(tables=None), INVALID),
                           (dict(chead=120), UNSUPPORTED), (dict(mask=P(4)), UNSUPPORTED),
                           (dict(ws=P(8)), UNSUPPORTED), (dict(rows=2049), UNSUPPORTED)):
        assert call(f, tree, **change) == status, change


def test_python_takes_no_null_scale(L):
    import quantization_amax_reduce_b200 as qar
    dev = torch.device("cpu")
    with pytest.raises(ValueError, match="null"):
        qar._scale3(0, "descale", True, dev)
    with pytest.raises(ValueError, match="takes no"):
        qar._scale3(0, "descale", False, dev)
    assert qar._scale3(64, "descale", True, dev) == 64
    C = qar._native()
    plain = lambda d: [x.value or 0 if isinstance(x, P) else 0 if x is None else x  # noqa: E731
                       for x in d.values()]
    assert C.write(*plain(dict(WRITE, qs=None))) == INVALID
    assert C.tree_fwd(*plain(dict(TREE, ds=None))) == INVALID
    # the bf16 calls take the same arguments, with no scale
    for f, good in ((C.write_bf16, dict(WRITE, qs=None, tokens=0)),
                    (C.tree_fwd_bf16, dict(TREE, ds=None, rows=0))):
        assert f(*plain(good)) == OK
        assert f(*plain(dict(good, dim=64))) == UNSUPPORTED
        assert f(*plain(dict(good, num=0))) == INVALID
        with pytest.raises(TypeError, match="number of arguments"):
            f(*plain(good)[:-1])
    for f, good in ((C.write_bf16, WRITE), (C.tree_fwd_bf16, TREE)):
        with pytest.raises(ValueError, match="no scale"):
            f(*plain(good))


def test_shares_of_the_work_list_up_to_its_limit(tmp_path):
    """The calls take bounds of up to 2^31 - 1 work items: a CTA's share of them
    may not overflow on the way (the compiler refuses a constant that does)."""
    import os
    import subprocess
    from quantization_amax_reduce_b200 import build
    source = "#include \"kernels.h\"\nusing fp8attn::tree_items_per_cta;\n"
    cases = [(0, 1, 4), (0, 148, 4), (1, 148, 4), (4, 1, 4), (592, 148, 4), (593, 148, 5),
             (740, 148, 5), (741, 148, 6), (5, 1, 5)]
    cases += [(t, n, -(-t // n)) for t in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 148, 2 ** 31 - 149)
              for n in (1, 2, 147, 148)]
    for total, ctas, want in cases:
        source += f"static_assert(tree_items_per_cta({total}, {ctas}) == {want}, \"\");\n"
    (tmp_path / "share.cpp").write_text(source)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    r = subprocess.run(["g++", "-std=c++17", "-fsyntax-only", "-w", "-I", build.CSRC, "-I", cuda,
                        str(tmp_path / "share.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[:2000]


def test_stall_self_test_checks_its_arguments(L):
    for which, tile in ((-1, 0), (2, 0), (0, -1)):
        assert L.fp8attn_selftest_kv_tree_stall(which, tile) == INVALID


def test_build_without_pythons_headers(tmp_path, monkeypatch):
    """The library is built where Python's headers are missing, as before there
    was a CPython module beside it; what needs the module says so."""
    import os
    import subprocess
    import quantization_amax_reduce_b200 as qar
    from quantization_amax_reduce_b200 import build
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfp8attn.so"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})

    def compiler(cmd, **kw):
        if build.CALLS_SRC in cmd and not os.path.exists(tmp_path / "Python.h"):
            raise subprocess.CalledProcessError(1, cmd)
        target = cmd[cmd.index("-o") + 1]
        if target.startswith(str(tmp_path)):
            open(target, "w").close()

    monkeypatch.setattr(build.subprocess, "check_call", compiler)
    with pytest.warns(UserWarning, match="Python.h"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)
    (tmp_path / "Python.h").write_text("")
    build.build()
    assert os.path.exists(build.CALLS)

    def no_module(*a):
        raise ImportError("no _calls")

    monkeypatch.setattr(qar, "_native_calls", None)
    monkeypatch.setattr(qar.importlib, "import_module", no_module)
    with pytest.raises(RuntimeError, match="_calls module is missing"):
        qar._native()
