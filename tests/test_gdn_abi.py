"""The gated delta layer's C ABI and binding on the CPU: exports and refusals, all
before any HIP call."""
import ctypes
import math
import os
import re

import pytest

import nvfp4_w4a4_block_quantize_amd as nv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nvfp4_gdn.h")
OK, NULL, SHAPE, ALIGN, DTYPE, RANGE, DEVICE = range(7)
P = 1 << 20  # a fake, aligned "device" address: validation never dereferences it
BIG = 1 << 31


def declared_functions():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*nvfp4_status\s*(nvfp4_\w+)\s*\(", src, flags=re.M)))


@pytest.fixture(scope="module")
def lib():
    path = os.environ.get("NVFP4_GDN_ABI_LIB")  # another build of the C ABI layer (the sanitized host build)
    if path:
        found = ctypes.CDLL(path)
        for name, (res, args) in nv.GDN_SIGNATURES.items():
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
    assert declared_functions() == sorted(nv.GDN_SIGNATURES)
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

    conv = dict(channels=80, width=4, dtype=1, x=P, ldx=80, weight=P, bias=None, act=1, slots=P, state=P, state_out=P, n_slots=5,
                out=2 * P, ldo=80, stream=None)
    delta = dict(hk=2, hv=4, dk=128, dv=64, dtype=1, q=P, qt=256, qh=128, k=P, kt=256, kh=128, v=P, vt=256, vh=64, a=P, at=4, b=P, bt=4,
                 a_log=P, dt=P, scale=0.1, eps=1e-6, slots=P, state=P, state_out=P, n_slots=5, out=2 * P, ot=256, oh=64, stream=None)
    heads = "hk hv dk dv dtype q qt qh k kt kh v vt vh a at b bt a_log dt scale eps"
    return {
        "conv": caller("nvfp4_causal_conv", "tokens channels width dtype x ldx weight bias act n starts cached slots state state_out n_slots "
                       "out ldo stream", dict(tokens=9, n=3, starts=P, cached=P, **conv)),
        "conv_step": caller("nvfp4_causal_conv_step", "n channels width dtype x ldx weight bias act slots state state_out n_slots out ldo "
                            "stream", dict(n=3, **conv)),
        "chunked": caller("nvfp4_gated_delta_chunked", f"tokens {heads} n starts cached slots state state_out n_slots out ot oh ws bytes "
                          "stream", dict(tokens=9, n=3, starts=P, cached=P, ws=P, bytes=1 << 40, **delta)),
        "step": caller("nvfp4_gated_delta_step", f"n {heads} slots state state_out n_slots out ot oh stream", dict(n=3, **delta)),
        "norm": caller("nvfp4_group_norm", "tokens groups dim dtype x xt xg weight wg bias gate gt gg act centred eps out ot og stream",
                       dict(tokens=9, groups=4, dim=24, dtype=1, x=P, xt=96, xg=24, weight=P, wg=0, bias=P, gate=3 * P, gt=96, gg=24, act=1,
                            centred=1, eps=1e-6, out=2 * P, ot=96, og=24, stream=None)),
    }


CONV = ([(NULL, k, None) for k in "x weight slots state state_out out".split()]
        + [(DTYPE, "dtype", 3), (DTYPE, "dtype", -1), (DTYPE, "act", 2), (SHAPE, "channels", 0), (SHAPE, "channels", (1 << 26) + 1),
           (SHAPE, "width", 1), (SHAPE, "width", 5), (SHAPE, "n", 0), (SHAPE, "n", BIG - 1), (SHAPE, "n_slots", 0), (SHAPE, "n_slots", BIG),
           (SHAPE, "ldx", 79), (SHAPE, "ldo", 79), (SHAPE, "ldx", 1 << 40), (SHAPE, "out", P)]
        + [(ALIGN, k, P + 1) for k in "x out state state_out".split()] + [(ALIGN, k, P + 2) for k in "weight bias slots".split()])
DELTA = ([(NULL, k, None) for k in "q k v a b a_log dt slots state state_out out".split()]
         + [(DTYPE, "dtype", 5), (RANGE, "scale", 0.0), (RANGE, "scale", -1.0), (RANGE, "scale", math.inf), (RANGE, "scale", math.nan),
            (RANGE, "eps", -1e-9), (RANGE, "eps", math.nan), (RANGE, "eps", math.inf), (SHAPE, "hk", 0), (SHAPE, "hk", 3), (SHAPE, "hv", 0),
            (SHAPE, "hv", 1 << 33), (SHAPE, "dk", 96), (SHAPE, "dk", 32), (SHAPE, "dv", 0), (SHAPE, "dv", 96), (SHAPE, "dv", 320),
            (SHAPE, "n", 0), (SHAPE, "n", BIG - 1), (SHAPE, "n_slots", 0), (SHAPE, "n_slots", BIG), (SHAPE, "qt", 248), (SHAPE, "kh", 64),
            (SHAPE, "vt", 248), (SHAPE, "oh", 32), (SHAPE, "at", 3), (SHAPE, "bt", 3), (SHAPE, "vt", 1 << 40), (SHAPE, "at", 1 << 40),
            (SHAPE, "out", P)]
         + [(ALIGN, k, 2 * P + 8) for k in "q k v out state state_out".split()] + [(ALIGN, "a", P + 1), (ALIGN, "b", P + 1)]
         + [(ALIGN, k, s) for k, s in (("qt", 260), ("kt", 260), ("vt", 260), ("ot", 260))] + [(ALIGN, k, P + 2) for k in "a_log dt slots".split()])
REFUSED = {
    "conv": CONV + [(NULL, "starts", None), (SHAPE, "tokens", 0), (SHAPE, "tokens", BIG), (ALIGN, "starts", P + 1), (ALIGN, "cached", P + 2)],
    "conv_step": CONV,
    "chunked": DELTA + [(NULL, "starts", None), (NULL, "ws", None), (SHAPE, "tokens", 0), (SHAPE, "tokens", BIG), (SHAPE, "bytes", 15),
                        (SHAPE, "bytes", -1), (ALIGN, "ws", P + 8), (ALIGN, "starts", P + 1), (ALIGN, "cached", P + 2)],
    "step": DELTA,
    "norm": [(NULL, k, None) for k in "x weight out".split()]
    + [(DTYPE, "dtype", 3), (DTYPE, "act", 2), (DTYPE, "act", -1), (DTYPE, "centred", 2), (RANGE, "eps", -1.0), (RANGE, "eps", math.nan),
       (SHAPE, "tokens", 0), (SHAPE, "tokens", BIG), (SHAPE, "groups", 0), (SHAPE, "groups", 1 << 26), (SHAPE, "dim", 0), (SHAPE, "dim", 8193),
       (SHAPE, "xt", 95), (SHAPE, "xg", 23), (SHAPE, "gt", 95), (SHAPE, "ot", 95), (SHAPE, "og", 25), (SHAPE, "wg", 23), (SHAPE, "wg", -24),
       (SHAPE, "xt", 1 << 40), (ALIGN, "x", P + 1), (ALIGN, "gate", P + 1), (ALIGN, "out", P + 1), (ALIGN, "weight", P + 2),
       (ALIGN, "bias", P + 2)],
}


@pytest.mark.parametrize("op", sorted(REFUSED))
def test_refusals(lib, op):
    call = calls(lib)[op]
    for status, name, value in REFUSED[op]:
        assert call(**{name: value}) == status, (name, value)


def test_in_place_norm_wants_the_same_strides(lib):
    call = calls(lib)["norm"]
    assert call(out=P, ot=192) == SHAPE and call(out=P, og=32, ot=128) == SHAPE
    assert call(out=3 * P, gt=192) == SHAPE


def test_products_of_sizes_past_32_bits(lib):
    c = calls(lib)
    assert c["chunked"](tokens=BIG - 1, hv=128, vt=1 << 16, ot=1 << 16, at=128, bt=128) == SHAPE
    assert c["step"](n=BIG - 2, hv=128, vt=1 << 16, ot=1 << 16, at=128, bt=128) == SHAPE
    assert c["step"](n=(1 << 26) + 1) == SHAPE and c["chunked"](n=(1 << 26) + 1) == SHAPE  # 4 value heads each
    assert c["step"](hk=1 << 25, hv=1 << 25) == SHAPE


def test_heads_lie_within_their_token(lib):
    """Tensors laid out by heads first, which do not overlap either, are refused, as the header says."""
    c = calls(lib)
    assert c["norm"](xt=24, xg=9 * 24) == SHAPE and c["norm"](ot=24, og=9 * 24) == SHAPE and c["norm"](gt=24, gg=9 * 24) == SHAPE
    for name in ("step", "chunked"):
        assert c[name](qt=128, qh=9 * 128) == SHAPE and c[name](kt=128, kh=9 * 128) == SHAPE
        assert c[name](vt=64, vh=9 * 64) == SHAPE and c[name](ot=64, oh=9 * 64) == SHAPE
    assert "token >= (heads - 1) *" in open(HEADER).read()


def test_strides_whose_products_pass_64_bits(lib):
    """Heads by a head's stride, up to 2^26 by 2^40: what wraps to a small or negative number overlaps all the same."""
    c = calls(lib)
    many = (1 << 25) + 1
    for token, group in ((1, 1 << 39), (1, (1 << 40) - 1), (many, 1 << 39), ((1 << 40) - 1, (1 << 40) - 1), ((1 << 40) - 1, 1 << 38)):
        for row in ("x", "o", "g"):
            rows = dict(xt=many, xg=1, ot=many, og=1, gt=many, gg=1)
            rows[row + "t"], rows[row + "g"] = token, group
            assert c["norm"](groups=many, dim=1, wg=0, **rows) == SHAPE, (row, token, group)
    for heads in (2, 3, 1 << 19):  # of 128
        far = (1 << 40) - 8
        assert c["step"](hk=heads, hv=heads, dk=128, dv=128, vt=heads * 128, vh=128, ot=heads * 128, oh=128, qt=heads * 128, qh=128, kt=far, kh=far,
                         at=heads, bt=heads) == SHAPE


def test_valid_calls_without_a_gpu_return_device_error(lib):
    if not no_gpu():
        pytest.skip("a GPU is visible: valid calls would launch kernels on these placeholder addresses")
    for name, call in calls(lib).items():
        assert call() == DEVICE, name
    c = calls(lib)
    assert c["conv"](cached=None, bias=P, x=P + 2, ldx=81) == DEVICE  # element alignment is enough
    assert c["chunked"](cached=None, a=P + 2, at=5, state_out=3 * P) == DEVICE
    assert c["norm"](gate=None, bias=None, wg=24, out=P, x=P) == DEVICE
    assert c["norm"](gate=2 * P) == DEVICE  # out = gate


def test_workspace_size(lib):
    size = ctypes.c_int64(-1)
    call, at = lib.nvfp4_gated_delta_workspace, ctypes.addressof(size)
    assert call(8, 1, 2, 4, 128, 128, 1, None) == NULL
    assert call(8, 1, 2, 4, 128, 128, 9, at) == DTYPE
    for bad in ((0, 1, 2, 4, 128, 128), (8, 0, 2, 4, 128, 128), (BIG, 1, 2, 4, 128, 128), (8, 1, 3, 4, 128, 128), (8, 1, 2, 4, 96, 128),
                (8, 1, 2, 4, 128, 100), (BIG - 1, 1, 2, 128, 128, 128)):
        assert call(*bad, 1, at) == SHAPE and size.value == -1, bad
    sizes = []
    for tokens, n in ((1, 1), (64, 1), (65, 1), (8192, 1), (8192, 40), (BIG - 1, 40)):
        assert call(tokens, n, 8, 48, 128, 128, 1, at) == OK
        sizes.append(size.value)
    assert sizes == sorted(sizes) and sizes[0] > 0 and all(s % 16 == 0 for s in sizes)


def test_binding_refuses_bad_tensors():
    torch = pytest.importorskip("torch")
    i32 = dict(dtype=torch.int32)
    x, weight, state = torch.zeros((9, 80)), torch.zeros((80, 4)), torch.zeros((5, 3, 80))
    slots, starts = torch.zeros(3, **i32), torch.zeros(4, **i32)
    good = dict(x=x, weight=weight, state=state, slots=slots, token_starts=starts, cached_lens=slots, bias=torch.zeros(80))
    bad_conv = (({"x": x[0]}, "x must be"), ({"x": x.t()}, "unit column"), ({"weight": weight[:79]}, "weight must be"),
                ({"weight": weight.half()}, "weight must be"), ({"bias": torch.zeros(79)}, "bias must be"), ({"state": state[:, :2]}, "state must be"),
                ({"state": state.half()}, "state must be"), ({"state_out": state[:4]}, "state_out must be"),
                ({"state": torch.zeros((3, 5, 80)).transpose(0, 1)}, "contiguous"), ({"out": x.half()}, "out must be"),
                ({"activation": "gelu"}, "activation"), ({"slots": slots.long()}, "slots must be"))
    for change, match in bad_conv + (({"token_starts": slots}, "token_starts must"), ({"cached_lens": starts}, "cached_lens must")):
        with pytest.raises(ValueError, match=match):
            nv.nvfp4_causal_conv(**{**good, **change})
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_causal_conv(**good)
    step = {k: v for k, v in good.items() if k not in ("token_starts", "cached_lens")}
    step["slots"] = torch.zeros(9, **i32)
    for change, match in bad_conv[:-1] + (({"slots": slots}, "slots must have shape"),):
        with pytest.raises(ValueError, match=match):
            nv.nvfp4_causal_conv_step(**{**step, **change})
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_causal_conv_step(**step)

    q, v, a, per = torch.zeros((9, 2, 64)), torch.zeros((9, 4, 128)), torch.zeros((9, 4)), torch.zeros(4)
    good = dict(q=q, k=q.clone(), v=v, a=a, b=a, a_log=per, dt_bias=per, state=torch.zeros((5, 4, 64, 128)), slots=slots, token_starts=starts,
                workspace=torch.zeros(64, dtype=torch.uint8))
    bad = (({"k": q[:, :1]}, "k must be"), ({"k": q.half()}, "k must be"), ({"v": v[:8], "a": a, "out": v[:8]}, "v must have 9"),
           ({"v": v.half()}, "v must be|out must be"), ({"a": a[:, :3]}, "a must be"), ({"b": a.half()}, "b must be"),
           ({"a": torch.zeros((4, 9)).t()}, "unit column"), ({"a_log": per[:3]}, "a_log must"), ({"dt_bias": per.double()}, "dt_bias must"),
           ({"state": torch.zeros((5, 4, 128, 64))}, "state must be"), ({"state_out": torch.zeros((4, 4, 64, 128))}, "state_out must be"),
           ({"out": v.half()}, "out must be"), ({"q": q.transpose(1, 2)}, "q must have unit stride|k must be"))
    for change, match in bad + (({"workspace": torch.zeros(64)}, "workspace must be"), ({"token_starts": slots}, "token_starts must")):
        with pytest.raises(ValueError, match=match):
            nv.nvfp4_gated_delta_chunked(**{**good, **change})
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_gated_delta_chunked(**good)
    step = {k: t for k, t in good.items() if k not in ("token_starts", "workspace")}
    step["slots"] = torch.zeros(9, **i32)
    for change, match in bad + (({"slots": slots}, "slots must have shape"),):
        with pytest.raises(ValueError, match=match):
            nv.nvfp4_gated_delta_step(**{**step, **change})
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_gated_delta_step(**step)

    x = torch.zeros((9, 4, 24))
    good = dict(x=x, weight=torch.zeros(24), bias=torch.zeros(24), gate=x.clone())
    for change, match in (({"x": x[0]}, "x must be"), ({"weight": torch.zeros(23)}, "weight must be"), ({"weight": torch.zeros((4, 24))}, "bias must be"),
                          ({"bias": torch.zeros((4, 24))}, "bias must be"), ({"gate": x.half()}, "gate must be"), ({"gate": x[:8]}, "gate must be"),
                          ({"out": x[:, :3]}, "out must be"), ({"x": x.transpose(1, 2)}, "unit stride"), ({"activation": 3}, "activation")):
        with pytest.raises(ValueError, match=match):
            nv.nvfp4_group_norm(**{**good, **change})
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_group_norm(**good)
    with pytest.raises(TypeError, match="unsupported dtype"):
        nv.nvfp4_group_norm(x.double(), torch.zeros(24))


def test_binding_refuses_tensors_of_other_dimensions():
    """Before any size of them is read, with a workspace given or not."""
    torch = pytest.importorskip("torch")
    q, v, a, per = torch.zeros((9, 2, 64)), torch.zeros((9, 4, 128)), torch.zeros((9, 4)), torch.zeros(4)
    good = dict(q=q, k=q.clone(), v=v, a=a, b=a, a_log=per, dt_bias=per, state=torch.zeros((5, 4, 64, 128)),
                slots=torch.zeros(3, dtype=torch.int32), token_starts=torch.zeros(4, dtype=torch.int32))
    for change in ({"q": q[0]}, {"q": q[0, 0, 0]}, {"v": v[0]}, {"v": v.view(9, 4, 2, 64)}, {"slots": good["slots"][0]},
                   {"slots": good["slots"].view(1, 3)}):
        for workspace in (None, torch.zeros(64, dtype=torch.uint8)):
            with pytest.raises(ValueError, match="must be"):
                nv.nvfp4_gated_delta_chunked(**{**good, **change}, workspace=workspace)
    step = {k: t for k, t in good.items() if k != "token_starts"}
    for change in ({"q": q[0, 0, 0]}, {"q": q[0]}, {"v": v[0]}):
        with pytest.raises(ValueError, match="must be"):
            nv.nvfp4_gated_delta_step(**{**step, **change, "slots": torch.zeros(9, dtype=torch.int32)})
