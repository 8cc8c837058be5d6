"""The paged KV cache's C ABI and binding on the CPU: exports, refusals (all
before any HIP call), and the exactness of the division that the kernels use."""
import ctypes
import math
import os
import random
import re

import pytest

import nvfp4_w4a4_block_quantize_amd as nv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nvfp4_kv.h")
OK, NULL, SHAPE, ALIGN, DTYPE, RANGE, DEVICE = range(7)
P = 1 << 20  # a fake, aligned "device" address: validation never dereferences it


def declared_functions():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*nvfp4_status\s*(nvfp4_\w+)\s*\(", src, flags=re.M)))


@pytest.fixture(scope="module")
def lib():
    path = os.environ.get("NVFP4_KV_ABI_LIB")  # another build of the C ABI layer (the sanitized host build)
    if path:
        found = ctypes.CDLL(path)
        for name, (res, args) in nv.KV_SIGNATURES.items():
            getattr(found, name).restype, getattr(found, name).argtypes = res, args
        return found
    if not os.path.exists(nv.LIB_PATH):
        pytest.skip("libnvfp4.so not built")
    return nv.load_library()


def no_gpu():
    if os.environ.get("NVFP4_NO_GPU") == "1":
        return True
    torch = pytest.importorskip("torch")
    return torch.cuda.device_count() == 0


def test_every_declared_symbol_is_exported_and_bound(lib):
    assert declared_functions() == sorted(nv.KV_SIGNATURES)
    for name in declared_functions():
        assert hasattr(lib, name) and callable(getattr(nv, name))


def calls(lib):
    """Each entry point as a function of its arguments by name, all of them valid."""
    def caller(name, order, valid):
        def call(**kw):
            assert set(kw) <= set(valid), kw
            a = {**valid, **kw}
            return getattr(lib, name)(*[a[k] for k in order.split()])
        return call

    table = caller("nvfp4_kv_block_table",
                   "n cached new page free n_free used table max_pages ld slots tokens lens starts first used_out stream",
                   dict(n=4, cached=P, new=P, page=16, free=P, n_free=10, used=P, table=P, max_pages=8, ld=8, slots=P,
                        tokens=64, lens=P, starts=P, first=P, used_out=P, stream=None))
    rope = caller("nvfp4_rope",
                  "tokens dim rot dtype adjacent pos axes_n ld_pos freq axes q qo hq qt qh qot qoh k ko hk kt kh kot koh stream",
                  dict(tokens=4, dim=64, rot=32, dtype=1, adjacent=0, pos=P, axes_n=3, ld_pos=4, freq=P, axes=P, q=P, qo=2 * P,
                       hq=8, qt=512, qh=64, qot=512, qoh=64, k=P, ko=2 * P, hk=2, kt=128, kh=64, kot=128, koh=64, stream=None))
    write = caller("nvfp4_kv_cache_write", "tokens heads dim dtype k kt kh v vt vh ks vs slots ck cv pages page stream",
                   dict(tokens=4, heads=2, dim=64, dtype=1, k=P, kt=128, kh=64, v=P, vt=128, vh=64, ks=P, vs=P, slots=P,
                        ck=P, cv=2 * P, pages=8, page=16, stream=None))
    attend = caller("nvfp4_paged_attention",
                    "n hq hk dim dtype q qt qh ck cv pages page ks vs table max_pages ld lens scale window out ot oh lse ws bytes "
                    "stream",
                    dict(n=4, hq=8, hk=2, dim=64, dtype=1, q=P, qt=512, qh=64, ck=P, cv=2 * P, pages=8, page=16, ks=P, vs=P,
                         table=P, max_pages=8, ld=8, lens=P, scale=0.125, window=0, out=2 * P, ot=512, oh=64, lse=None, ws=P,
                         bytes=1 << 28, stream=None))
    return {"table": table, "rope": rope, "write": write, "attend": attend}


BIG = 1 << 31
REFUSED = {
    "table": [(NULL, k, None) for k in "cached new free used table slots lens starts first used_out".split()]
    + [(SHAPE, "n", 0), (SHAPE, "n", -1), (SHAPE, "n", BIG), (SHAPE, "page", 0), (SHAPE, "page", 12), (SHAPE, "page", 1032),
       (SHAPE, "n_free", -1), (SHAPE, "n_free", BIG), (SHAPE, "max_pages", 0), (SHAPE, "max_pages", 9), (SHAPE, "tokens", 0),
       (SHAPE, "tokens", BIG), (SHAPE, "ld", 1 << 41)]
    + [(ALIGN, k, P + 2) for k in "cached new free used table slots lens starts first used_out".split()],
    "rope": [(NULL, k, None) for k in "pos freq axes q qo k ko".split()]
    + [(DTYPE, "dtype", 3), (DTYPE, "dtype", -1), (DTYPE, "adjacent", 2), (SHAPE, "tokens", 0), (SHAPE, "tokens", BIG),
       (SHAPE, "dim", 0), (SHAPE, "dim", 63), (SHAPE, "rot", 0), (SHAPE, "rot", 31), (SHAPE, "rot", 66), (SHAPE, "axes_n", 0),
       (SHAPE, "axes_n", 9), (SHAPE, "ld_pos", 3), (SHAPE, "hq", 0), (SHAPE, "hq", 1 << 27), (SHAPE, "hk", -1),
       (SHAPE, "qt", 511), (SHAPE, "qh", 63), (SHAPE, "qoh", 65), (SHAPE, "kot", 127), (SHAPE, "kt", 1 << 41),
       (ALIGN, "q", P + 1), (ALIGN, "ko", P + 1), (ALIGN, "pos", P + 2), (ALIGN, "axes", P + 1), (ALIGN, "freq", P + 3)],
    "write": [(NULL, k, None) for k in "k v ks vs slots ck cv".split()]
    + [(DTYPE, "dtype", 7), (SHAPE, "tokens", 0), (SHAPE, "heads", 0), (SHAPE, "dim", 60), (SHAPE, "dim", -8),
       (SHAPE, "pages", 0), (SHAPE, "pages", BIG // 16), (SHAPE, "page", 20), (SHAPE, "page", 2048), (SHAPE, "kt", 120),
       (SHAPE, "vh", 56), (SHAPE, "cv", P), (ALIGN, "k", P + 8), (ALIGN, "v", P + 8), (ALIGN, "kt", 132), (ALIGN, "ks", P + 2),
       (ALIGN, "slots", P + 1), (ALIGN, "ck", P + 8)],
    "attend": [(NULL, k, None) for k in "q ck cv ks vs table lens out ws".split()]
    + [(DTYPE, "dtype", 5), (RANGE, "scale", 0.0), (RANGE, "scale", -1.0), (RANGE, "scale", math.inf), (RANGE, "scale", math.nan),
       (SHAPE, "n", 0), (SHAPE, "hq", 0), (SHAPE, "hq", 7), (SHAPE, "hk", 3), (SHAPE, "dim", 96), (SHAPE, "dim", 32),
       (SHAPE, "window", -1), (SHAPE, "pages", 0), (SHAPE, "pages", BIG // 16), (SHAPE, "page", 4), (SHAPE, "max_pages", 9),
       (SHAPE, "max_pages", 0), (SHAPE, "out", P), (SHAPE, "qt", 448), (SHAPE, "oh", 32), (SHAPE, "bytes", 1024), (SHAPE, "bytes", -1),
       (ALIGN, "q", P + 8), (ALIGN, "out", P + 4), (ALIGN, "qt", 516), (ALIGN, "ck", P + 8), (ALIGN, "lse", P + 2),
       (ALIGN, "ws", P + 8), (ALIGN, "table", P + 1), (ALIGN, "lens", P + 2), (ALIGN, "vs", P + 1)],
}


@pytest.mark.parametrize("op", sorted(REFUSED))
def test_refusals(lib, op):
    call = calls(lib)[op]
    for status, name, value in REFUSED[op]:
        assert call(**{name: value}) == status, (name, value)


def test_in_place_rope_wants_the_same_strides(lib):
    call = calls(lib)["rope"]
    assert call(qo=P, qot=1024) == SHAPE
    assert call(ko=P, koh=64, kot=256) == SHAPE


def test_strides_whose_products_pass_64_bits(lib):
    """Heads by a head's stride, up to 2^25 by 2^40: what wraps to a small or negative number overlaps all the same."""
    call = calls(lib)["rope"]
    for heads, stride in (((1 << 24) + 1, (1 << 40) - 1), (1 << 25, 1 << 39), (1 << 25, (1 << 40) - 2)):
        for row in ("q", "qo", "k", "ko"):
            rows = {r + s: n for r in ("q", "qo", "k", "ko") for s, n in (("t", 2 * heads), ("h", 2))}
            rows[row + "h"], rows[row + "t"] = stride, 2
            assert call(dim=2, rot=2, hq=heads, hk=heads, **rows) == SHAPE, (row, heads, stride)


def test_pages_of_a_long_table_and_cache(lib):
    """Products of sizes that pass 32 bits are seen as what they are."""
    c = calls(lib)
    assert c["table"](max_pages=1 << 28, ld=1 << 28, page=1024) == SHAPE
    assert c["attend"](max_pages=1 << 28, ld=1 << 28, page=16) == SHAPE
    assert c["attend"](hq=1 << 33, hk=1) == SHAPE
    assert c["attend"](n=1 << 28) == SHAPE  # 8 query heads each
    long = dict(max_pages=1 << 24, ld=1 << 24, page=16)  # 2^28 tokens
    assert c["attend"](hq=1024, qt=1 << 16, ot=1 << 16, **long) == SHAPE
    assert c["attend"](hq=512, qt=1 << 15, ot=1 << 15, n=1 << 22, **long) == SHAPE
    assert c["write"](heads=1 << 25, dim=1 << 25) == SHAPE


def test_valid_calls_without_a_gpu_return_device_error(lib):
    if not no_gpu():
        pytest.skip("a GPU is visible: valid calls would launch kernels on these placeholder addresses")
    for name, call in calls(lib).items():
        assert call() == DEVICE, name
    c = calls(lib)
    assert c["table"](free=None, n_free=0) == DEVICE
    assert c["rope"](hk=0, k=None, ko=None) == DEVICE
    assert c["rope"](qo=P, ko=P) == DEVICE
    assert c["rope"](q=P + 2, qt=513) == DEVICE  # element alignment is enough
    assert c["attend"](lse=P, window=5) == DEVICE


def test_workspace_size(lib):
    size = ctypes.c_int64(-1)
    call = lib.nvfp4_paged_attention_workspace
    at = ctypes.addressof(size)
    assert call(8, 2, 64, None) == NULL
    for bad in ((7, 2, 64), (8, 0, 64), (0, 2, 64), (8, 2, 80)):
        assert call(*bad, at) == SHAPE and size.value == -1
    sizes = []
    for heads in ((2, 2), (24, 4), (32, 2), (64, 1)):
        assert call(*heads, 256, at) == OK
        sizes.append(size.value)
    assert sizes == sorted(sizes) and sizes[0] > 0 and all(s % 16 == 0 for s in sizes)
    assert sizes[-1] <= 1 << 27


def test_fast_division_is_exact(lib):
    if not os.environ.get("NVFP4_KV_ABI_LIB"):
        pytest.skip("the division is reached through the host build")
    div = lib.kv_test_fastdiv
    div.restype, div.argtypes = ctypes.c_uint32, [ctypes.c_uint32, ctypes.c_uint32]
    rng = random.Random(1)
    most = BIG - 1
    for d in list(range(1, 1100)) + [rng.randrange(1, most) for _ in range(500)] + [most, most - 1, 1 << 30, (1 << 30) + 1]:
        top = most // d
        near = [q * d + r for q in (0, 1, 2, top - 1, top, rng.randrange(top + 1)) for r in (-1, 0, 1, d - 1)]
        for n in near + [most, rng.randrange(most)]:
            if 0 <= n <= most:
                assert div(d, n) == n // d, (d, n)


def test_binding_refuses_bad_tensors():
    torch = pytest.importorskip("torch")
    i32 = dict(dtype=torch.int32)
    lens, table, slots = torch.zeros(4, **i32), torch.zeros((4, 8), **i32), torch.zeros(64, **i32)
    one, free = torch.zeros(1, **i32), torch.zeros(10, **i32)
    args = dict(cached_lens=lens, new_lens=lens, page_size=16, free_pages=free, free_used=one, block_table=table, slot_map=slots)
    for name, value, match in (("new_lens", lens[:3], "new_lens must have shape"), ("new_lens", lens.long(), "must be int32"),
                               ("block_table", table[:3], "block_table must be int32"), ("block_table", table.t()[:4], "must be int32|unit column"),
                               ("free_used", free, "free_used must have shape"), ("slot_map", slots.view(8, 8), "must be 1-D"),
                               ("slot_map", slots[::2], "slot_map must be contiguous")):
        with pytest.raises(ValueError, match=match):
            nv.nvfp4_kv_block_table(**{**args, name: value})
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_kv_block_table(**args)

    q, k = torch.zeros((5, 8, 64)), torch.zeros((5, 2, 64))
    pos, freq, axes = torch.zeros((3, 5), **i32), torch.zeros(16), torch.zeros(16, **i32)
    for change, match in (({"positions": pos[:, :4]}, "positions must be"), ({"positions": pos.long()}, "positions must be"),
                          ({"inv_freq": freq.double()}, "inv_freq must be"), ({"axes": axes[:3]}, "axes must have shape"),
                          ({"k": k.half()}, "k must be"), ({"k": k[:4]}, "k must be"), ({"q_out": q.half()}, "q_out must be"),
                          ({"k": None, "k_out": k}, "k_out without k"), ({"q": q.transpose(1, 2)}, "unit stride")):
        with pytest.raises(ValueError, match=match):
            nv.nvfp4_rope(**{**dict(q=q, k=k, positions=pos, inv_freq=freq, axes=axes), **change})
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_rope(q, k, pos, freq, axes)

    scale, cache = torch.ones(1), torch.zeros((6, 2, 16, 64), dtype=torch.uint8)
    good = dict(k=k, v=k, k_scale=scale, v_scale=scale, slot_map=torch.zeros(5, **i32), k_cache=cache, v_cache=cache.clone())
    for change, match in (({"v": k[:, :1]}, "v must be"), ({"k_scale": torch.ones(2)}, "k_scale must be"),
                          ({"slot_map": slots}, "slot_map must have shape"), ({"k_cache": cache.int()}, "k_cache must be uint8"),
                          ({"v_cache": cache[:5]}, "v_cache must have shape"), ({"k_cache": cache[:, :1].contiguous(), "v_cache": cache[:, :1].contiguous()}, "k_cache must be"),
                          ({"k_cache": cache[0]}, "k_cache must be")):
        with pytest.raises(ValueError, match=match):
            nv.nvfp4_kv_cache_write(**{**good, **change})
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_kv_cache_write(**good)

    good = dict(q=q, k_cache=cache, v_cache=cache.clone(), k_scale=scale, v_scale=scale, block_table=torch.zeros((5, 4), **i32),
                seq_lens=torch.zeros(5, **i32))
    for change, match in (({"q": q[:, :, :32]}, "head_dim"), ({"block_table": table}, "block_table must be"), ({"seq_lens": lens}, "seq_lens must have"),
                          ({"lse": torch.zeros((5, 7))}, "lse must be"), ({"lse": torch.zeros((5, 8)).double()}, "lse must be"),
                          ({"out": q.half()}, "out must be"), ({"workspace": torch.zeros(4)}, "workspace must be")):
        with pytest.raises(ValueError, match=match):
            nv.nvfp4_paged_attention(**{"workspace": torch.zeros(16, dtype=torch.uint8), **good, **change})
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_paged_attention(**good)
