"""Host-only checks of include/moe_kv8.h's entry points and their Python
objects: every refusal has its status and its reason, and nothing is launched
(no GPU is touched)."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

from moe_expert_layer_warp_gb300 import api, batch, build

ONE = 1 << 20          # stands for an aligned device pointer; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


def _why():
    return api.load().moe_last_cuda_error_string().decode()


# ------------------------------------------------------------------ rotary --
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923,
              10 ** 64)


@pytest.mark.parametrize("radians", [
    [1.0, 0.5, 1e-4, 1e-9, 0.0, 6.283185307179586, 7.5, 1e6, 2.0 ** 40],
    [-1.0, -1e-4, -7.5, 1e-300, -1e-300, 3.141592653589793], []])
def test_turns(lib, radians):
    got = api.moe_rotary_turns(radians)
    assert got.dtype is torch.int64 and got.shape == (len(radians),)
    for f, t in zip(radians, got.tolist()):
        off = (t - round(Fraction(f) / (2 * PI) * 2 ** 64)) % 2 ** 64
        # a turn's 2^-64, and the product's own rounding for many turns
        assert min(off, 2 ** 64 - off) <= 2 + abs(f) * 2.0 ** -40


@pytest.mark.parametrize("bad", [math.nan, math.inf, 1e13])
def test_turns_refusals(lib, bad):
    with pytest.raises(api.MoeError):
        api.moe_rotary_turns([1.0, bad])
    assert "finite" in _why()
    assert lib.moe_rotary_turns(None, -1, None) == api.MOE_EINVAL
    assert lib.moe_rotary_turns(None, 1, None) == api.MOE_EINVAL


def _rotary(**over):
    f = dict(head_dim=128, n_rotated=64, first=0, interleaved=0, amplitude=1.0, turns=ONE)
    f.update(over)
    return api.RotaryDesc(*[f[n] for n, _ in api.RotaryDesc._fields_])


def _rows(**over):
    f = dict(in_=ONE, out=ONE + 4096, n_heads=4, in_token_stride=512, in_head_stride=128,
             out_token_stride=512, out_head_stride=128)
    f.update(over)
    return api.RotaryRows(*[f[n] for n, _ in api.RotaryRows._fields_])


@pytest.mark.parametrize("over,status,reason", [
    (dict(head_dim=0), api.MOE_EINVAL, "within a head"),
    (dict(n_rotated=0), api.MOE_EINVAL, "within a head"),
    (dict(first=-8), api.MOE_EINVAL, "within a head"),
    (dict(first=72), api.MOE_EINVAL, "within a head"),
    (dict(n_rotated=144), api.MOE_EINVAL, "within a head"),
    (dict(interleaved=2), api.MOE_EINVAL, "interleaved"),
    (dict(amplitude=math.inf), api.MOE_EINVAL, "amplitude"),
    (dict(turns=None), api.MOE_EINVAL, "turns"),
    (dict(turns=ONE + 4), api.MOE_EINVAL, "turns"),
    (dict(n_rotated=24), api.MOE_EUNSUPPORTED, "multiples of 16"),
    (dict(head_dim=2048), api.MOE_EUNSUPPORTED, "multiples of 16"),
    (dict(head_dim=120), api.MOE_EUNSUPPORTED, "multiples of 16"),
    (dict(first=4), api.MOE_EUNSUPPORTED, "multiples of 16"),
])
def test_rotary_descriptor_refusals(lib, over, status, reason):
    d, r = _rotary(**over), _rows()
    assert lib.moe_rotary(ctypes.byref(d), api.MOE_BF16, ctypes.byref(r), None, ONE, 3,
                          None) == status
    assert reason in _why()


@pytest.mark.parametrize("over,reason", [
    (dict(n_heads=-1), "n_heads"), (dict(in_=None), "null"), (dict(out=ONE + 8), "aligned"),
    (dict(in_token_stride=500), "strides"), (dict(in_head_stride=-128), "strides"),
    (dict(out_head_stride=1 << 40), "strides"), (dict(out_token_stride=256), "overlap"),
    (dict(out_head_stride=64), "overlap"), (dict(out_token_stride=0), "overlap"),
    (dict(out=ONE, in_token_stride=1024), "in place"), (dict(n_heads=40000, out_token_stride=1 << 30),
                                                        "n_heads")])
def test_rotary_rows_refusals(lib, over, reason):
    d, good, r = _rotary(), _rows(), _rows(**over)
    for q, k in ((r, None), (good, r)):
        assert lib.moe_rotary(ctypes.byref(d), api.MOE_BF16, ctypes.byref(q),
                              None if k is None else ctypes.byref(k), ONE, 3,
                              None) == api.MOE_EINVAL
        assert reason in _why()


def test_rotary_other_refusals(lib):
    d, r = ctypes.byref(_rotary()), ctypes.byref(_rows())
    f = lib.moe_rotary
    assert f(None, api.MOE_BF16, r, r, ONE, 3, None) == api.MOE_EINVAL
    assert f(d, 5, r, r, ONE, 3, None) == api.MOE_EINVAL and "type" in _why()
    assert f(d, api.MOE_BF16, r, r, ONE, -1, None) == api.MOE_EINVAL and "n_tokens" in _why()
    assert f(d, api.MOE_BF16, r, r, None, 3, None) == api.MOE_EINVAL and "positions" in _why()
    assert f(d, api.MOE_BF16, r, r, ONE + 2, 3, None) == api.MOE_EINVAL and "positions" in _why()
    # memory that one writes and the other has
    for over in (dict(), dict(in_=ONE + 8192), dict(in_=ONE + 4096, out=ONE + 8192),
                 dict(in_=ONE + 8192, out=ONE)):
        other = ctypes.byref(_rows(**over))
        assert f(d, api.MOE_BF16, r, other, ONE, 3, None) == api.MOE_EINVAL
        assert "share memory" in _why()
    # nothing to do: no token, no rows
    assert f(d, api.MOE_BF16, r, r, None, 0, None) == api.MOE_OK
    assert f(d, api.MOE_BF16, None, None, ONE, 3, None) == api.MOE_OK


@pytest.mark.parametrize("args", [dict(n_rotated=63), dict(n_rotated=64, base=0.0),
                                  dict(n_rotated=64, scaling="longer"),
                                  dict(n_rotated=64, scaling="linear", factor=0.0),
                                  dict(n_rotated=2, scaling="base", factor=2.0),
                                  dict(n_rotated=64, scaling="ramp", base=1.0),
                                  dict(n_rotated=64, fast=1.0, slow=1.0),
                                  dict(n_rotated=64, original=0)])
def test_frequencies_refusals(args):
    with pytest.raises(ValueError):
        batch.rotary_frequencies(**args)


def test_frequencies():
    plain = batch.rotary_frequencies(64)
    assert plain[0] == 1.0 and abs(plain[16] - 1e-2) < 1e-16 and len(plain) == 32
    assert batch.rotary_frequencies(64, scaling="linear", factor=4.0) == [v / 4 for v in plain]
    base = batch.rotary_frequencies(64, scaling="base", factor=4.0)
    assert base[0] == 1.0 and abs(base[31] / (plain[31] / 4) - 1) < 1e-12
    for kind in ("ramp", "bands"):
        f = batch.rotary_frequencies(64, scaling=kind, factor=8.0, original=4096, fast=32.0,
                                     slow=1.0)
        ratio = [a / b for a, b in zip(f, plain)]
        assert ratio == sorted(ratio, reverse=True)
        for r, v in zip(ratio, plain):
            turns = 4096 * v / (2 * math.pi)
            assert 1 / 8 - 1e-12 <= r <= 1 + 1e-12
            if turns > 45:                       # beyond the next pair's
                assert abs(r - 1) < 1e-12
            if turns < 0.7:
                assert abs(r - 1 / 8) < 1e-12
    # bands: in between by the number of turns itself
    f = batch.rotary_frequencies(64, scaling="bands", factor=8.0, fast=4.0, slow=1.0)
    for a, v in zip(f, plain):
        w = min(1.0, max(0.0, (4096 * v / (2 * math.pi) - 1.0) / 3.0))
        assert abs(a - (w * v + (1 - w) * v / 8)) <= 1e-15 * v


# ------------------------------------------------------------------- cache --
def _cache(**over):
    f = dict(k=ONE, v=ONE, k_scale=ONE, v_scale=ONE, n_pages=10, page_size=32, n_kv_heads=2,
             head_dim=64, block=16, page_stride=32 * 128, token_stride=128, head_stride=64)
    f.update(over)
    return api.Kv8CacheC(*[f[n] for n, _ in api.Kv8CacheC._fields_])


CACHE_FAULTS = [
    (dict(k=None), api.MOE_EINVAL, "aligned"),
    (dict(v=ONE + 8), api.MOE_EINVAL, "aligned"),
    (dict(k_scale=None), api.MOE_EINVAL, "scales"),
    (dict(v_scale=ONE + 2), api.MOE_EINVAL, "scales"),
    (dict(n_pages=0), api.MOE_EINVAL, "n_pages"),
    (dict(n_pages=1 << 31), api.MOE_EINVAL, "n_pages"),
    (dict(n_kv_heads=0), api.MOE_EINVAL, "sizes"),
    (dict(n_kv_heads=1 << 15), api.MOE_EINVAL, "sizes"),
    (dict(token_stride=120), api.MOE_EINVAL, "strides"),
    (dict(head_stride=0), api.MOE_EINVAL, "strides"),
    (dict(page_stride=1 << 40), api.MOE_EINVAL, "stride out of range"),
    (dict(page_size=8), api.MOE_EUNSUPPORTED, "page_size"),
    (dict(page_size=48), api.MOE_EUNSUPPORTED, "page_size"),
    (dict(page_size=512), api.MOE_EUNSUPPORTED, "page_size"),
    (dict(block=8), api.MOE_EUNSUPPORTED, "block"),
    (dict(block=64), api.MOE_EUNSUPPORTED, "block"),
    (dict(block=24), api.MOE_EUNSUPPORTED, "block"),
    (dict(head_dim=96), api.MOE_EUNSUPPORTED, "head_dim"),
]


@pytest.mark.parametrize("over,status,reason", CACHE_FAULTS)
def test_cache_refusals(lib, over, status, reason):
    c, a = ctypes.byref(_cache(**over)), api.AttnDesc(8, 0, 0, 0.125)
    assert lib.moe_kv8_append(c, ONE, ONE, api.MOE_BF16, 128, 64, 3, ONE, None) == status
    assert reason in _why() and "moe_kv8_append" in _why()
    assert lib.moe_kv8_read(c, ONE, 3, api.MOE_BF16, ONE, ONE + 64, 128, 64, None) == status
    assert reason in _why() and "moe_kv8_read" in _why()
    assert lib.moe_attend8_workspace_bytes(c, ctypes.byref(a)) == 0
    assert lib.moe_attend8(c, ctypes.byref(a), api.MOE_BF16, ONE, 512, 64, 4, ONE, ONE, ONE, 4, 2,
                           ONE, 1 << 30, ONE, 512, 64, None) == status
    assert reason in _why() and "moe_attend8" in _why()


@pytest.mark.parametrize("at,value,reason", [
    (0, None, "null"), (1, ONE + 8, "misaligned"), (2, 3, "type"), (3, 100, "strides"),
    (4, -64, "strides"), (4, 1 << 40, "strides"), (5, -1, "n_tokens"), (6, None, "slots"),
    (6, ONE + 4, "misaligned")])
def test_append_refusals(lib, at, value, reason):
    args = [ONE, ONE, api.MOE_BF16, 128, 64, 3, ONE]
    args[at] = value
    assert lib.moe_kv8_append(ctypes.byref(_cache()), *args, None) == api.MOE_EINVAL
    assert reason in _why()


@pytest.mark.parametrize("over", [dict(v=ONE, v_scale=ONE + 4096),
                                  dict(v=ONE + 4096, v_scale=ONE)])
def test_append_refuses_keys_and_values_in_one_place(lib, over):
    c = _cache(k=ONE, k_scale=ONE, **over)
    assert lib.moe_kv8_append(ctypes.byref(c), ONE, ONE, api.MOE_BF16, 128, 64, 3, ONE,
                              None) == api.MOE_EINVAL
    assert "share memory" in _why()


@pytest.mark.parametrize("at,value,reason", [
    (0, None, "null"), (0, ONE + 4, "misaligned"), (1, -1, "n out"), (2, 3, "type"),
    (3, None, "null"), (4, ONE, "the same"), (5, 100, "strides"), (5, 64, "overlap"),
    (6, 32, "overlap"), (6, 0, "overlap")])
def test_read_refusals(lib, at, value, reason):
    args = [ONE, 3, api.MOE_BF16, ONE, ONE + 4096, 128, 64]
    args[at] = value
    assert lib.moe_kv8_read(ctypes.byref(_cache()), *args, None) == api.MOE_EINVAL
    assert reason in _why()


def test_nothing_to_do(lib):
    c = ctypes.byref(_cache())
    assert lib.moe_kv8_append(c, None, None, api.MOE_F32, 128, 64, 0, None, None) == api.MOE_OK
    assert lib.moe_kv8_read(c, None, 0, api.MOE_F32, None, None, 128, 64, None) == api.MOE_OK


# --------------------------------------------------------------- attention --
@pytest.mark.parametrize("desc,status,reason", [
    ((7, 0, 0, 0.1), api.MOE_EINVAL, "multiple"), ((0, 0, 0, 0.1), api.MOE_EINVAL, "multiple"),
    ((8, -1, 0, 0.1), api.MOE_EINVAL, "window"), ((8, 4, -1, 0.1), api.MOE_EINVAL, "window"),
    ((8, 0, 0, 0.0), api.MOE_EINVAL, "scale"), ((8, 0, 0, math.nan), api.MOE_EINVAL, "scale"),
    ((130, 0, 0, 0.1), api.MOE_EUNSUPPORTED, "64 query heads")])
def test_attend_descriptor_refusals(lib, desc, status, reason):
    c, a = ctypes.byref(_cache()), api.AttnDesc(*desc)
    assert lib.moe_attend8_workspace_bytes(c, ctypes.byref(a)) == 0
    assert lib.moe_attend8(c, ctypes.byref(a), api.MOE_BF16, ONE, 512, 64, 4, ONE, ONE, ONE, 4, 2,
                           ONE, 1 << 30, ONE, 512, 64, None) == status
    assert reason in _why()


@pytest.mark.parametrize("at,value,reason", [
    (0, api.MOE_F32, "bf16 or fp16"), (0, 9, "bf16 or fp16"), (1, ONE + 8, "q or out"),
    (1, None, "q or out"), (2, 100, "q strides"), (3, 0, "q strides"), (4, -1, "n_tokens"),
    (5, None, "q_start"), (6, ONE + 2, "misaligned"), (7, None, "block_table"),
    (8, 0, "max_blocks"), (9, 0, "n_requests"), (9, 1025, "n_requests"), (10, None, "workspace"),
    (10, ONE + 16, "workspace"), (11, 16, "workspace"), (12, ONE + 8, "q or out"),
    (13, 100, "out strides"), (13, 256, "out strides"), (14, 32, "out strides")])
def test_attend_refusals(lib, at, value, reason):
    c, a = _cache(), api.AttnDesc(8, 0, 0, 0.125)
    for f in (lib.moe_attend8, lib.moe_attend8_padded):
        args = [api.MOE_BF16, ONE, 512, 64, 4, ONE, ONE, ONE, 4, 2, ONE, 1 << 30, ONE, 512, 64]
        args[at] = value
        assert f(ctypes.byref(c), ctypes.byref(a), *args, None) == api.MOE_EINVAL
        assert reason in _why()


def test_binding_refuses_tensors_of_another_kind(lib):
    """What the calls cannot see: types and shapes behind the pointers. (None of
    these tensors is on a GPU; each refusal comes before that is asked.)"""
    codes = torch.zeros(3, 32, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.ones(3, 2, 2)
    assert api.make_cache8(codes, codes, scale, scale).block == 16
    for args, reason in [
            ((codes, codes[:2], scale, scale), "one shape"),
            ((codes.float(), codes.float(), scale, scale), "float8_e4m3fn"),
            ((codes, codes.float(), scale, scale), "float8_e4m3fn"),
            ((codes, codes, scale.double(), scale), "k_scale"),
            ((codes, codes, scale, scale[:2]), "v_scale"),
            ((codes, codes, scale, torch.ones(3, 2, 1)), "v_scale"),
            ((codes, codes, torch.ones(3, 2, 3), torch.ones(3, 2, 3)), "k_scale"),
            ((codes, codes, scale.transpose(1, 2), scale), "k_scale")]:
        with pytest.raises(ValueError, match=reason):
            api.make_cache8(*args)
    c, a = _cache(), api.AttnDesc(8, 0, 0, 0.125)
    B16, I32 = torch.bfloat16, torch.int32
    q, ws = torch.zeros(4, 8, 64, dtype=B16), torch.zeros(16, dtype=torch.uint8)
    start, length, table = (torch.zeros(n, dtype=I32) for n in (3, 2, 8))
    table = table.view(2, 4)
    good = dict(q=q, q_start=start, kv_len=length, block_table=table, workspace=ws, out=q)
    for over, reason in [
            (dict(q=q.float(), out=q.float()), "bfloat16 or float16"),
            (dict(q=q[:, :7], out=q[:, :7]), "q"), (dict(out=q[:3]), "out"),
            (dict(out=q.half()), "out"), (dict(q_start=start[:2]), "q_start"),
            (dict(kv_len=length.long()), "kv_len"), (dict(block_table=table[0]), "block_table"),
            (dict(q=q.transpose(0, 2).contiguous().transpose(0, 2)), "contiguous")]:
        for padded in (False, True):
            with pytest.raises(ValueError, match=reason):
                api.moe_attend8(c, a, **dict(good, **over), padded=padded)
    k, slots = torch.zeros(4, 2, 64, dtype=B16), torch.zeros(4, dtype=torch.int64)
    for args, reason in [((k[:, :1], k[:, :1], slots), "k must"), ((k, k.float(), slots), "v must"),
                         ((k, k, slots[:3]), "slots"), ((k, k, slots.int()), "slots"),
                         ((k.double(), k.double(), slots), "float32"),
                         ((k, k.transpose(0, 1).contiguous().transpose(0, 1), slots), "strides")]:
        with pytest.raises(ValueError, match=reason):
            api.moe_kv8_append(c, *args)
    for args, reason in [((slots.int(), k, k), "slots"), ((slots, k[:3], k[:3]), "k must"),
                         ((slots, k, k.half()), "v must"),
                         ((slots, k.double(), k.double()), "float32")]:
        with pytest.raises(ValueError, match=reason):
            api.moe_kv8_read(c, *args)
    d, pos = _rotary(head_dim=64), torch.zeros(4, dtype=I32)
    for args, reason in [((q[:3], None, pos), "q must"), ((None, q[..., :32], pos), "k must"),
                         ((q, q.half(), pos), "one type"), ((q.double(), None, pos), "one type"),
                         ((None, None, pos), "give q or k"), ((q, None, pos.long()), "positions"),
                         ((q, None, pos, q[:, :7]), "out must")]:
        with pytest.raises(ValueError, match=reason):
            api.moe_rotary(d, *args)


def test_objects_refuse_what_they_cannot_hold(lib):
    with pytest.raises(ValueError, match="CUDA"):
        codes = torch.zeros(3, 32, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
        batch.PagedCache8(codes, codes, torch.ones(3, 2, 2), torch.ones(3, 2, 2))
    with pytest.raises(ValueError, match="block"):
        batch.PagedCache8.allocate(3, 32, 2, 64, block=48)
    with pytest.raises(ValueError, match="frequencies"):
        batch.Rotary(64, 32, frequencies=[1.0] * 15)
