"""Host-side checks of the attention calls (no GPU needed): every refusal of
the C ABI comes back before anything is enqueued, and the binding refuses
what it cannot describe to the library."""

import ctypes as C
import math

import pytest
import torch

import lut_binary_gemv_b200 as fb
from lut_binary_gemv_b200 import build as fb_build

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE, CUDA = range(6)
FAKE = 0x10000   # aligned and never dereferenced by a call that is refused
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    fb_build.build()
    return fb.lib()


def heads(**over):
    h = dict(q=FAKE, k=FAKE, v=FAKE, t=BF16, T=4, Hq=8, Hkv=2, D=128, ldq=1024, ldk=256, ldv=256)
    h.update(over)
    return fb.FbHeadsStruct(**h)


def kv_cache(**over):
    c = dict(k=FAKE, v=FAKE, t=BF16, pages=10, page_size=16, Hkv=2, D=128)
    c.update(over)
    return fb.FbKvCacheStruct(**c)


def rope(L, hin=None, hout=None, pos=FAKE, inv=FAKE, rot=128, wq=FAKE, wk=FAKE, eps=1e-6, cache=True, slots=FAKE,
         flags=0):
    hin, hout = hin or heads(), hout or heads()
    kv = kv_cache() if cache is True else cache
    return L.fb_qk_norm_rope(C.byref(hin), C.byref(hout), pos, inv, rot, wq, wk, eps,
                             None if kv is None else C.byref(kv), slots, flags, None)


@pytest.mark.parametrize("args,status", [
    (dict(hin=heads(q=None)), INVALID), (dict(hin=heads(k=None)), INVALID), (dict(hin=heads(v=None)), INVALID),
    (dict(hin=heads(T=0)), INVALID), (dict(hin=heads(T=(1 << 24) + 1)), INVALID), (dict(hin=heads(t=7)), INVALID),
    (dict(hin=heads(Hkv=3)), INVALID), (dict(hin=heads(Hkv=0)), INVALID), (dict(hin=heads(Hq=2000)), INVALID),
    (dict(hin=heads(ldq=1016)), INVALID), (dict(hin=heads(ldk=128)), INVALID), (dict(hin=heads(ldv=0)), INVALID),
    (dict(hout=heads(T=5)), INVALID), (dict(hout=heads(Hq=4)), INVALID), (dict(hout=heads(D=64)), INVALID),
    (dict(hout=heads(ldq=1000)), INVALID), (dict(hout=heads(ldk=8)), INVALID),
    (dict(pos=None), INVALID), (dict(inv=None), INVALID), (dict(rot=-16), INVALID), (dict(rot=144), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(slots=None), INVALID), (dict(cache=kv_cache(Hkv=1)), INVALID), (dict(cache=kv_cache(D=64)), INVALID),
    (dict(cache=kv_cache(t=F16)), INVALID), (dict(cache=kv_cache(page_size=24)), INVALID),
    (dict(cache=kv_cache(page_size=2048)), INVALID), (dict(cache=kv_cache(pages=0)), INVALID),
    (dict(cache=kv_cache(pages=1 << 27)), INVALID), (dict(cache=kv_cache(k=None)), INVALID),
    (dict(flags=2), INVALID), (dict(flags=0x20), INVALID),
    (dict(hout=heads(t=F32), cache=None, slots=None), UNSUPPORTED), (dict(rot=24), UNSUPPORTED),
    (dict(hin=heads(D=120, ldq=960, ldk=240, ldv=240), hout=heads(D=120, ldq=960, ldk=240, ldv=240), rot=112,
          cache=None), UNSUPPORTED),
    (dict(hin=heads(D=272, ldq=2176, ldk=544, ldv=544), hout=heads(D=272, ldq=2176, ldk=544, ldv=544),
          cache=None), UNSUPPORTED),
    (dict(hin=heads(q=FAKE + 8)), MISALIGNED), (dict(hin=heads(ldk=260)), MISALIGNED),
    (dict(hout=heads(v=FAKE + 2)), MISALIGNED), (dict(hout=heads(ldq=1028)), MISALIGNED),
    (dict(pos=FAKE + 2), MISALIGNED), (dict(inv=FAKE + 4), MISALIGNED), (dict(wq=FAKE + 1), MISALIGNED),
    (dict(slots=FAKE + 2), MISALIGNED), (dict(cache=kv_cache(v=FAKE + 8)), MISALIGNED),
])
def test_rope_refusals(L, args, status):
    assert rope(L, **args) == status


# in: q at 1 MB, k at 2 MB, v at 3 MB; rows of 2048, 512 and 512 bytes (bf16)
MB = 1 << 20


@pytest.mark.parametrize("args", [
    dict(hout=heads(q=MB, k=None, v=None, ldq=1032)),                       # in place with another pitch
    dict(hout=heads(q=MB, k=None, v=None, t=F16), cache=kv_cache(t=F16)),   # ... with another type
    dict(hin=heads(q=MB, k=2 * MB, v=3 * MB, t=F32), hout=heads(q=MB, k=None, v=None)),
    dict(hout=heads(q=None, k=None, v=2 * MB)),                             # an output that is another input
    dict(hout=heads(q=2 * MB, k=None, v=None)),
    dict(hin=heads(q=MB, k=2 * MB, v=2 * MB), hout=heads(q=None, k=2 * MB, v=None)),   # keys that are the values too
    dict(hout=heads(q=MB + 16, k=None, v=None)),                            # a part of its input
    dict(hout=heads(q=MB - 2048 * 4 + 16, k=None, v=None)),
    dict(hout=heads(q=MB + 2048 * 3 + 2032, k=None, v=None)),
    dict(hout=heads(q=None, k=2 * MB + 512, v=None)),                       # its input one row on
    dict(hout=heads(q=None, k=8 * MB, v=8 * MB)),                           # two outputs in one place
    dict(hout=heads(q=8 * MB, k=8 * MB + 2048 * 3, v=None)),
    dict(hin=heads(q=MB, k=MB + 2048, v=MB + 2560, ldq=1536, ldk=1536, ldv=1536),     # slices of one projection
         hout=heads(q=MB + 16, k=None, v=None, ldq=1536)),
    dict(hin=heads(q=MB, k=MB + 2048, v=MB + 2560, ldq=1536, ldk=1536, ldv=1536),
         hout=heads(q=None, k=MB + 2560, v=None, ldk=1536)),
])
def test_rope_refuses_outputs_that_overlap(L, args):
    assert rope(L, **{"hin": heads(q=MB, k=2 * MB, v=3 * MB), **args}) == INVALID


OUT = 0x20000


def prompt(L, h=None, cu=FAKE, n=2, scale=0.1, out=OUT, ldo=1024, lse=FAKE, flags=0):
    h = h or heads()
    return L.fb_attn_prompt(C.byref(h), cu, n, scale, out, ldo, lse, flags, None)


@pytest.mark.parametrize("args,status", [
    (dict(h=heads(q=None)), INVALID), (dict(h=heads(k=None)), INVALID), (dict(h=heads(v=None)), INVALID),
    (dict(h=heads(T=0)), INVALID), (dict(h=heads(Hkv=5)), INVALID), (dict(h=heads(ldq=512)), INVALID),
    (dict(cu=None), INVALID), (dict(n=0), INVALID), (dict(out=None), INVALID), (dict(ldo=1016), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-0.1), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(flags=2), INVALID), (dict(flags=0x10), INVALID),
    (dict(scale=2e38), INVALID), (dict(out=FAKE), INVALID),
    (dict(h=heads(t=F32)), UNSUPPORTED), (dict(h=heads(D=96)), UNSUPPORTED),
    (dict(h=heads(q=FAKE + 8)), MISALIGNED), (dict(h=heads(ldv=260)), MISALIGNED), (dict(out=OUT + 8), MISALIGNED),
    (dict(ldo=1028), MISALIGNED), (dict(cu=FAKE + 1), MISALIGNED), (dict(lse=FAKE + 2), MISALIGNED),
])
def test_prompt_refusals(L, args, status):
    assert prompt(L, **args) == status


def tree(L, q=FAKE, ldq=1024, T=4, Hq=8, cache=None, table=FAKE, width=80, ld=80, lens=FAKE, cu=FAKE, n=2, most=3,
         mask=FAKE, scale=0.1, out=OUT, ldo=1024, lse=FAKE, ws=FAKE, ws_bytes=1 << 30, flags=0):
    kv = cache or kv_cache()
    return L.fb_attn_tree(q, ldq, T, Hq, C.byref(kv), table, width, ld, lens, cu, n, most, mask, scale, out, ldo, lse,
                          ws, ws_bytes, flags, None)


@pytest.mark.parametrize("args,status", [
    (dict(q=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(out=None), INVALID),
    (dict(T=0), INVALID), (dict(Hq=7), INVALID), (dict(Hq=0), INVALID), (dict(n=0), INVALID), (dict(n=65537), INVALID),
    (dict(cu=None), INVALID), (dict(most=0), INVALID), (dict(most=65), INVALID), (dict(width=0), INVALID),
    (dict(ld=79), INVALID), (dict(ldq=1016), INVALID), (dict(ldo=8), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(flags=2), INVALID), (dict(cache=kv_cache(t=F32)), INVALID),
    (dict(cache=kv_cache(page_size=0)), INVALID), (dict(cache=kv_cache(v=None)), INVALID),
    (dict(cache=kv_cache(D=96), ldq=1024), UNSUPPORTED),
    (dict(out=FAKE), INVALID), (dict(scale=math.inf), INVALID),
    (dict(q=FAKE + 8), MISALIGNED), (dict(out=OUT + 4), MISALIGNED), (dict(ldq=1028), MISALIGNED),
    (dict(table=FAKE + 2), MISALIGNED), (dict(lens=FAKE + 1), MISALIGNED), (dict(cu=FAKE + 2), MISALIGNED),
    (dict(mask=FAKE + 4), MISALIGNED), (dict(lse=FAKE + 1), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 8), WORKSPACE), (dict(ws_bytes=0), WORKSPACE),
])
def test_tree_refusals(L, args, status):
    assert tree(L, **args) == status


def test_tree_workspace_bytes(L):
    def size(Hq=64, most=1, width=100, **over):
        c = kv_cache(**{**dict(Hkv=8, page_size=64), **over})
        return L.fb_attn_tree_workspace_bytes(Hq, C.byref(c), most, width)
    sizes = [size(most=m) for m in (1, 2, 4, 5, 64)]
    assert 0 < sizes[0] == sizes[1] < sizes[2] < sizes[3] == sizes[4]    # up to 16, 32 and more rows a key head
    assert size(D=64) < sizes[0]
    assert size(most=64, page_size=4) < sizes[4]                         # small pages: 64 rows at a time
    assert size(width=8) == size(page_size=1, width=512) == 0 < size(width=9)   # short tables are not split
    assert size(most=64, width=8) == sizes[4]
    for bad in (dict(Hq=0), dict(Hq=2048), dict(Hq=63), dict(most=0), dict(most=65), dict(width=0), dict(D=96),
                dict(page_size=3), dict(k=None), dict(t=F32)):
        assert size(**bad) == 0
    assert L.fb_attn_tree_workspace_bytes(8, None, 1, 1) == 0


def test_tree_refuses_a_workspace_that_is_too_small(L):
    for page, most in ((16, 1), (16, 64), (4, 64)):
        c = kv_cache(Hkv=8, page_size=page)
        size = L.fb_attn_tree_workspace_bytes(64, C.byref(c), most, 1000)
        args = dict(q=FAKE, ldq=8192, T=64, Hq=64, cache=c, width=1000, ld=1000, n=2, most=most, ldo=8192)
        assert tree(L, **args, ws_bytes=size - 1) == WORKSPACE
        assert tree(L, **args, ws=FAKE + 4, ws_bytes=size) == WORKSPACE
        assert tree(L, **args, ws=None, ws_bytes=size) == WORKSPACE


def test_errors_call_refuses_null(L):
    assert L.fb_attn_errors(None, 0) == INVALID


def test_struct_bytes_match_the_structs():
    assert fb._HEADS.size == C.sizeof(fb.FbHeadsStruct) and fb._CACHE.size == C.sizeof(fb.FbKvCacheStruct)
    h = fb.FbHeadsStruct(q=1, k=2, v=3, t=4, T=5, Hq=6, Hkv=7, D=8, ldq=9, ldk=10, ldv=11)
    assert bytes(h) == fb._HEADS.pack(*range(1, 12))
    c = fb.FbKvCacheStruct(k=1, v=2, t=3, pages=4, page_size=5, Hkv=6, D=7)
    assert bytes(c) == fb._CACHE.pack(*range(1, 8))


def test_binding_refuses_what_is_not_on_the_gpu_or_shaped_otherwise():
    q, k = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fb.fb_attn_prompt(q, k, k, cu)
    with pytest.raises(ValueError):
        fb.fb_qk_norm_rope(q, k, k, None, None)
    with pytest.raises(ValueError):
        fb.fb_attn_tree(q, (k, k), cu[None], cu)


class Sketch:
    """What the binding asks of a tensor on GPU 0, without the memory."""

    def __init__(self, shape, dtype, strides=None, device=0):
        self.shape, self.dtype, self._device = torch.Size(shape), dtype, device
        full = [math.prod(shape[i + 1:]) for i in range(len(shape))]
        self._strides = tuple(strides or full)
        self._plain = list(self._strides) == full
        self.device = torch.device("cuda", device)

    def get_device(self):
        return self._device

    def is_contiguous(self):
        return self._plain

    def stride(self):
        return self._strides

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return 2

    def data_ptr(self):
        return FAKE


class Recorder:
    """In the library's place: notes what reaches it, and on which device."""

    def __init__(self, current, sizes=None):
        self.calls, self._current, self._sizes = [], current, sizes or {}

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self._current[0], args))
            return self._sizes.get(name, 0)
        return call


@pytest.fixture
def sketched(monkeypatch):
    current = [0]
    recorder = Recorder(current)

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, current[0] = current[0], self.device

        def __exit__(self, *_):
            current[0] = self.before

    monkeypatch.setattr(fb, "lib", lambda: recorder)
    monkeypatch.setattr(fb, "_get_device", lambda: current[0])
    monkeypatch.setattr(fb, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: type("S", (), {"cuda_stream": 0}))
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: Sketch([shape] if isinstance(shape, int) else shape, dtype))
    recorder.current = current
    return recorder


@pytest.mark.parametrize("far", [2 ** 31, 2 ** 32 + 512])
def test_binding_refuses_pitches_past_32_bits(sketched, far):
    # the C ABI's pitches are ints: cut off, 2^32 + 512 would have passed for 512
    bf = torch.bfloat16
    h = lambda H, pitch=None: Sketch((2, H, 64), bf, pitch and (pitch, 64, 1))  # noqa: E731
    i32 = lambda *shape: Sketch(shape, torch.int32)  # noqa: E731
    q, kv, cu = h(8), h(2), i32(2)
    cache = (Sketch((4, 2, 16, 64), bf), Sketch((4, 2, 16, 64), bf))
    table, wide = i32(2, 4), Sketch((2, 4), torch.int32, (far, 1))
    for call in (lambda: fb.fb_attn_prompt(h(8, far), kv, kv, cu), lambda: fb.fb_attn_prompt(q, kv, h(2, far), cu),
                 lambda: fb.fb_attn_prompt(q, kv, kv, cu, out=h(8, far)),
                 lambda: fb.fb_attn_tree(h(8, far), cache, table, i32(2)),
                 lambda: fb.fb_attn_tree(q, cache, table, i32(2), out=h(8, far)),
                 lambda: fb.fb_attn_tree(q, cache, wide, i32(2)),
                 lambda: fb.fb_qk_norm_rope(q, h(2, far), kv, None, None),
                 lambda: fb.fb_qk_norm_rope(q, kv, kv, None, None, q_out=h(8, far))):
        with pytest.raises(ValueError):
            call()
    assert not [c for c in sketched.calls if not c[0].endswith("_bytes")]
    fb.fb_attn_tree(h(8, 2 ** 31 - 8), cache, Sketch((2, 4), torch.int32, (2 ** 31 - 1, 1)), i32(2))
    assert sketched.calls[-1][0] == "fb_attn_tree" and sketched.calls[-1][2][1] == 2 ** 31 - 8


@pytest.mark.parametrize("current", [0, 1])
def test_workspace_is_that_of_the_tensors_device(sketched, current):
    # its size goes by the SMs of the device that runs the call
    bf = torch.bfloat16
    sketched.current[0] = current
    sketched._sizes["fb_attn_tree_workspace_bytes"] = 64
    cache = tuple(Sketch((4, 2, 16, 64), bf, device=1) for _ in range(2))
    q, out, lens = Sketch((2, 8, 64), bf, device=1), Sketch((2, 8, 64), bf, device=1), Sketch((2,), torch.int32, device=1)
    assert fb.fb_attn_tree_workspace_bytes(8, cache, 1, 4) == 64
    fb.fb_attn_tree(q, cache, Sketch((2, 4), torch.int32, device=1), lens, out=out)
    assert [(name, device) for name, device, _ in sketched.calls] == [
        ("fb_attn_tree_workspace_bytes", 1), ("fb_attn_tree_workspace_bytes", 1), ("fb_attn_tree", 1)]
    assert sketched.calls[-1][2][-3] == 64 and sketched.current[0] == current


def test_rope_frequencies():
    f = fb.rope_frequencies(8, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64),
                                                       rtol=1e-14)
