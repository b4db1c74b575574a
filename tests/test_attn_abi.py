"""Host checks of the softmax layers' entry points (no GPU): sizes, and every
refusal before anything is enqueued."""
import ctypes

import numpy as np
import pytest

P = ctypes.c_void_p
D = P(0x10000)          # an aligned address that no refused call may touch


@pytest.fixture(scope="module")
def stq():
    import quantized_linear_attention_amd as q
    return q


@pytest.fixture(scope="module")
def L(stq):
    from quantized_linear_attention_amd import _lib
    return _lib._L


def kvd(**kw):
    from quantized_linear_attention_amd._lib import _KvDesc
    d = dict(n_blocks=10, block_tokens=64, n_kv_heads=2, d=128)
    d.update(kw)
    return _KvDesc(*[d[k] for k in ("n_blocks", "block_tokens", "n_kv_heads", "d")])


def nd(**kw):
    from quantized_linear_attention_amd._lib import _NormDesc
    d = dict(n_tok=3, n_q_heads=4, n_k_heads=2, d=128, in_type=0, out_type=0, norm=1, eps=1e-6, n_rot=64, rot_pairs=0,
             n_pos=10, q_stride=512, k_stride=256, q_out_stride=512, k_out_stride=256)
    d.update(kw)
    return _NormDesc(*[d[f[0]] for f in _NormDesc._fields_])


def ad(**kw):
    from quantized_linear_attention_amd._lib import _AttendDesc
    d = dict(n_req=3, n_tok=3, n_heads=4, type=0, table_cols=5, max_new=1, max_len=300, window=0, n_sink=0, scale=0.1,
             q_stride=512, o_stride=512)
    d.update(kw)
    return _AttendDesc(*[d[f[0]] for f in _AttendDesc._fields_])


def test_sizes(stq):
    # 64 tokens of one head at d = 128: 2 * 64 bytes of codes and 2 * 4 scale bytes each
    assert stq.stq_kv_bytes(10, 64, 2, 128) == 10 * 2 * 64 * (64 + 64 + 4 + 4)
    assert stq.stq_kv_bytes(3, 32, 1, 64) == 3 * 32 * 68
    assert stq.stq_kv_bytes(2 ** 31 - 1, 256, 8, 128) == (2 ** 31 - 1) * 8 * 256 * 136
    for bad in ((0, 64, 2, 128), (1, 16, 2, 128), (1, 48, 2, 128), (1, 512, 2, 128), (1, 64, 0, 128), (1, 64, 2, 96),
                (1, 64, 2, 256)):
        assert stq.stq_kv_bytes(*bad) == 0


def test_plan_refusals(L):
    def call(n=3, n_free=2, n_blocks=10, T=64, cols=4, n_tok=5, **null):
        p = dict(cached=D, new=D, free=D, table=D, tok=D, len=D, pos=D, slot=D, used=D)
        p.update(null)
        return L.stq_kv_plan(n, p["cached"], p["new"], p["free"], n_free, n_blocks, T, p["table"], cols, n_tok, p["tok"],
                             p["len"], p["pos"], p["slot"], p["used"], None)
    for kw in (dict(n=0), dict(n=-1), dict(n=4097), dict(n_free=-1), dict(n_blocks=0), dict(T=16), dict(T=100), dict(cols=0),
               dict(n_tok=-1)) + tuple({k: None} for k in ("cached", "new", "free", "table", "tok", "len", "pos", "slot", "used")):
        assert call(**kw) == -1, kw


def test_norm_refusals(L):
    def call(d, **null):
        p = dict(q=D, k=D, wq=None, wk=None, pos=D, cs=D, qo=P(0x20000), ko=P(0x30000))
        p.update(null)
        return L.stq_qk_norm_rope(ctypes.byref(d), p["q"], p["k"], p["wq"], p["wk"], p["pos"], p["cs"], p["qo"], p["ko"], None)
    for kw in (dict(n_tok=-1), dict(n_tok=(1 << 28) + 1), dict(n_q_heads=0), dict(n_k_heads=-1), dict(d=96), dict(d=32), dict(in_type=3), dict(out_type=1),
               dict(in_type=2, out_type=0), dict(norm=3), dict(norm=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(n_rot=8), dict(n_rot=-16), dict(n_rot=144), dict(rot_pairs=2), dict(n_pos=0)):
        assert call(nd(**kw)) == -1, kw
    for name in ("q", "k", "pos", "cs", "qo", "ko"):
        assert call(nd(), **{name: None}) == -1, name
    # layout: alignment, strides shorter than a token or off 16 bytes
    for kw in (dict(q_stride=508), dict(q_stride=514), dict(k_stride=255), dict(q_out_stride=516), dict(k_out_stride=0)):
        assert call(nd(**kw)) == -2, kw
    for name in ("q", "k", "wq", "wk", "cs", "qo", "ko"):
        assert call(nd(), **{name: P(0x10008)}) == -2, name
    # in place with another stride or type
    assert call(nd(q_out_stride=1024), qo=D) == -1
    assert call(nd(out_type=2), qo=D) == -1
    assert call(nd(n_tok=0), q=None) == 0
    assert L.stq_qk_norm_rope(None, D, D, None, None, D, D, D, D, None) == -1


def test_store_fetch_refusals(L):
    def store(d=None, cache=D, size=None, slot=D, n=3, k=D, v=D, ks=256, vs=256, ty=0):
        d = d or kvd()
        size = L.stq_kv_bytes(ctypes.byref(d)) if size is None else size
        return L.stq_kv_store(ctypes.byref(d), cache, size, slot, n, k, v, ks, vs, ty, None)
    for kw in (dict(d=kvd(d=96)), dict(d=kvd(block_tokens=33)), dict(d=kvd(n_blocks=0)), dict(n=-1), dict(ty=3), dict(ty=-1),
               dict(slot=None), dict(k=None), dict(v=None)):
        assert store(**kw) == -1, kw
    full = L.stq_kv_bytes(ctypes.byref(kvd()))
    for kw in (dict(cache=None), dict(cache=P(0x10004)), dict(size=full - 1), dict(k=P(0x10002)), dict(v=P(0x10008)),
               dict(ks=255), dict(ks=260), dict(vs=128), dict(ks=258, ty=2)):
        assert store(**kw) == -2, kw
    assert store(n=0, slot=None) == 0

    def fetch(cache=D, size=full, slot=D, n=3, k=D, v=D, ty=0):
        return L.stq_kv_fetch(ctypes.byref(kvd()), cache, size, slot, n, k, v, ty, None)
    for kw in (dict(n=-1), dict(ty=3), dict(slot=None), dict(k=None), dict(v=None)):
        assert fetch(**kw) == -1, kw
    for kw in (dict(cache=None), dict(size=full - 1), dict(k=P(0x10008)), dict(v=P(0x10004))):
        assert fetch(**kw) == -2, kw


def test_attend_refusals(L):
    kv = kvd()
    full = L.stq_kv_bytes(ctypes.byref(kv))

    def call(a=None, d=kv, size=full, work=P(0x40000), wbytes=1 << 40, **null):
        p = dict(cache=D, table=D, tok=D, len=D, q=D, o=P(0x20000))
        p.update(null)
        a = ad() if a is None else a
        return L.stq_kv_attend(ctypes.byref(d), p["cache"], size, ctypes.byref(a), p["table"], p["tok"], p["len"], p["q"],
                               p["o"], work, wbytes, None)
    for kw in (dict(n_req=-1), dict(n_tok=-1), dict(n_tok=(1 << 28) + 1), dict(n_heads=0), dict(n_heads=3), dict(n_heads=-2), dict(type=2), dict(type=-1),
               dict(table_cols=0), dict(table_cols=1 << 25), dict(max_new=0), dict(max_len=0), dict(window=-1), dict(n_sink=-1),
               dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(ad(**kw)) == -1, kw
    for name in ("table", "tok", "len", "q", "o"):
        assert call(**{name: None}) == -1, name
    assert call(d=kvd(d=32)) == -1
    for kw in (dict(q_stride=504), dict(o_stride=516)):
        assert call(ad(**kw)) == -2, kw
    for kw in (dict(cache=P(0x10008)), dict(q=P(0x10008)), dict(o=P(0x10002)), dict(size=full - 1)):
        assert call(**kw) == -2, kw
    # a call whose work is split takes a workspace of the stated size
    big = ad(max_len=4096)
    need = L.stq_kv_attend_bytes(ctypes.byref(kv), ctypes.byref(big))
    assert need > 0
    assert call(big, work=None) == -2 and call(big, wbytes=need - 1) == -2 and call(big, work=P(0x40004)) == -2
    assert call(ad(n_req=0)) == 0 and call(ad(n_tok=0)) == 0
    # more workgroups than a grid holds
    assert call(ad(n_req=1 << 20, n_tok=4, max_new=1 << 20, q_stride=512)) == -5


class Fake:
    """Stands in for a CUDA tensor where there is no GPU: the binding's checks run first."""

    def __init__(self, shape, dtype, device="cuda:0", stride=None, ptr=0x10000):
        import torch
        self.shape, self.dtype, self.device, self.is_cuda = tuple(shape), dtype, torch.device(device), True
        st, acc = [], 1
        for n in reversed(self.shape):
            st.insert(0, acc)
            acc *= n
        self._st, self._ptr = tuple(stride or st), ptr
        self._dense = stride is None

    def is_contiguous(self):
        return self._dense

    def numel(self):
        return int(np.prod(self.shape))

    def stride(self):
        return self._st

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return self._ptr

    def get_device(self):
        return self.device.index


def test_binding_refusals(stq, monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)   # some refusals are the library's own
    b, f, i, l, u = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
    E = stq.StqError
    with pytest.raises(E, match="pages"):
        stq.make_kv(Fake([100], u), 64, 2, 128)
    with pytest.raises(E, match="pages"):
        stq.make_kv(Fake([1 << 20], f), 64, 2, 128)
    with pytest.raises(E, match="pages"):
        stq.make_kv(Fake([1 << 20], u), 64, 2, 96)
    kv = stq.make_kv(Fake([10 * 2 * 64 * 136 + 5], u), 64, 2, 128)
    assert kv.desc.n_blocks == 10
    k = Fake([4, 2, 128], b)
    s = Fake([4], l)
    for bad, what in ((dict(k=Fake([3, 2, 128], b)), "k is"), (dict(v=Fake([4, 1, 128], b)), "v is"),
                      (dict(v=Fake([4, 2, 64], b)), "v is"), (dict(slots=Fake([4], i)), "slots"),
                      (dict(v=Fake([4, 2, 128], f)), "one element type"), (dict(k=Fake([4, 2, 128], b, "cuda:1")), "cuda:1"),
                      (dict(k=Fake([4, 2, 128], b, stride=(512, 256, 1))), "contiguous"),
                      (dict(v=Fake([4, 2, 128], b, stride=(512, 128, 2))), "contiguous"),
                      (dict(k=Fake([4, 256], b)), "tokens"), (dict(k=None), "k must")):
        args = dict(slots=s, k=k, v=k)
        args.update(bad)
        with pytest.raises(E, match=what):
            stq.stq_kv_store(kv, stream=0, **args)
    for bad in (dict(k_out=Fake([4, 2, 127], b)), dict(v_out=Fake([4, 2, 128], f)), dict(slots=Fake([5], l)),
                dict(k_out=Fake([4, 2, 128], l), v_out=Fake([4, 2, 128], l))):
        args = dict(slots=s, k_out=k, v_out=k)
        args.update(bad)
        with pytest.raises(E):
            stq.stq_kv_fetch(kv, stream=0, **args)
    q = Fake([4, 6, 128], b)
    ok = dict(table=Fake([2, 5], i), tok_start=Fake([3], i), lens=Fake([2], i), q=q, o=q)
    for bad in (dict(table=Fake([10], i)), dict(table=Fake([2, 5], l)), dict(tok_start=Fake([2], i)), dict(lens=Fake([3], i)),
                dict(o=Fake([4, 6, 128], torch.float16)), dict(o=Fake([3, 6, 128], b)), dict(q=Fake([4, 6, 64], b)),
                dict(q=Fake([4, 6, 128], f), o=Fake([4, 6, 128], f)), dict(lens=Fake([2], i, "cuda:1")),
                dict(work=Fake([8], f)), dict(q=Fake([4, 6, 128], b, stride=(1536, 256, 1)))):
        args = dict(ok)
        args.update(bad)
        with pytest.raises(E):
            stq.stq_kv_attend(kv, scale=0.1, max_new=2, max_len=100, stream=0, **args)
    n = Fake([4, 6, 128], f)
    for bad in (dict(q_out=Fake([4, 6, 128], torch.float16)), dict(k_out=None), dict(k=Fake([3, 2, 128], b)),
                dict(k=Fake([4, 2, 128], f)), dict(q_weight=Fake([127], f)), dict(k_weight=Fake([128], b)),
                dict(cos_sin=Fake([9, 64], f)), dict(cos_sin=Fake([9 * 64], f), pos=Fake([4], i)),
                dict(cos_sin=Fake([9, 64], f), pos=Fake([5], i)), dict(cos_sin=Fake([9, 64], f), pos=Fake([4], l)),
                dict(q_out=n)):
        args = dict(q=q, k=k, q_out=Fake([4, 6, 128], b, ptr=0x20000), k_out=Fake([4, 2, 128], b, ptr=0x30000))
        args.update(bad)
        with pytest.raises(E):
            stq.stq_qk_norm_rope(stream=0, **args)
    for bad in (dict(max_new=2 ** 32 + 1), dict(max_len=2 ** 31), dict(window=2 ** 32), dict(n_sink=-2 ** 40)):
        args = dict(ok, max_new=2, max_len=100)
        args.update(bad)
        with pytest.raises(E, match="32 bits"):
            stq.stq_kv_attend(kv, scale=0.1, stream=0, **args)
    one = dict(cached=Fake([2], i), new=Fake([2], i), free=Fake([9], i), table=Fake([2, 5], i), block_tokens=64, n_blocks=10,
               tok_start=Fake([3], i), lens=Fake([2], i), pos=Fake([7], i), slots=Fake([7], l), used=Fake([1], i))
    for bad in (dict(cached=Fake([3], i)), dict(new=Fake([2], l)), dict(free=Fake([9], l)), dict(table=Fake([10], i)),
                dict(tok_start=Fake([2], i)), dict(slots=Fake([6], l)), dict(slots=Fake([7], i)), dict(used=Fake([2], i)),
                dict(table=Fake([3, 5], i)), dict(block_tokens=48), dict(n_blocks=0)):
        args = dict(one)
        args.update(bad)
        with pytest.raises(E):
            stq.stq_kv_plan(stream=0, **args)


def test_binding_passes_short_strides_on(stq, monkeypatch):
    """Tokens that overlap (one row expanded over the batch) keep their stride, which the library refuses."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    b, i, l, u = torch.bfloat16, torch.int32, torch.int64, torch.uint8
    kv = stq.make_kv(Fake([10 * 2 * 64 * 136], u), 64, 2, 128)
    good, flat = Fake([4, 2, 128], b), Fake([4, 2, 128], b, stride=(0, 128, 1))
    calls = [lambda x, y: stq.stq_kv_store(kv, Fake([4], l), x, y, stream=0),
             lambda x, y: stq.stq_kv_attend(kv, Fake([2, 5], i), Fake([3], i), Fake([2], i), x, y, 0.1, 2, 100, stream=0),
             lambda x, y: stq.stq_qk_norm_rope(x, None, y, None, stream=0)]
    for call in calls:
        for x, y in ((flat, good), (good, flat)):
            with pytest.raises(stq.StqError) as e:
                call(x, y)
            assert e.value.status in (-1, -2)       # before any launch


def test_plan_refuses_outputs_over_inputs(L):
    """Lengths written over the counts they come from, and any other output that reaches into an input."""
    at = {k: 0x100000 * (i + 1) for i, k in enumerate(("cached", "new", "free", "table", "tok", "len", "pos", "slot", "used"))}
    size = dict(cached=12, new=12, free=8, table=48, tok=16, len=12, pos=20, slot=40, used=4)

    def call(**over):
        p = {k: P(v) for k, v in dict(at, **over).items()}
        return L.stq_kv_plan(3, p["cached"], p["new"], p["free"], 2, 10, 64, p["table"], 4, 5, p["tok"], p["len"], p["pos"],
                             p["slot"], p["used"], None)
    for i in ("cached", "new", "free"):
        for o in ("table", "tok", "len", "pos", "slot", "used"):
            for a in (at[i], at[i] + size[i] - 4, at[i] - size[o] + 4):
                assert call(**{o: a}) == -1, (i, o)


def test_binding_refuses_values_a_descriptor_cannot_hold(stq, monkeypatch):
    import torch
    b, i = torch.bfloat16, torch.int32
    kv = stq.make_kv(Fake([10 * 2 * 64 * 136], torch.uint8), 64, 2, 128)
    q, o = Fake([4, 2, 128], b), Fake([4, 2, 128], b, ptr=0x20000)
    args = (kv, Fake([2, 5], i), Fake([3], i), Fake([2], i), q, o)
    for scale, max_new, window in (("1", 2, 0), (None, 2, 0), (0.1, 2.5, 0), (0.1, 2, 1.0)):
        with pytest.raises(stq.StqError, match="descriptor"):
            stq.stq_kv_attend(*args, scale, max_new, 100, window=window, stream=0)
    with pytest.raises(stq.StqError, match="descriptor"):
        stq.stq_qk_norm_rope(q, None, o, None, eps=None, stream=0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)   # an infinite scale is the library's to refuse
    for scale in (1e39, -1e39, float("nan")):
        with pytest.raises(stq.StqError) as e:
            stq.stq_kv_attend(*args, scale, 2, 100, stream=0)
        assert e.value.status == -1
    with pytest.raises(stq.StqError, match="descriptor"):
        stq.stq_kv_attend_bytes(kv, 2, 4, 2, 2, 100, window=3.5)


def test_packed_descriptors_are_the_structures():
    """The packed bytes lie as the structures' fields do."""
    import ctypes
    from quantized_linear_attention_amd import _lib
    for pack, desc in ((_lib._norm_desc, _lib._NormDesc), (_lib._attend_desc, _lib._AttendDesc)):
        values = [0.5 + i if t is ctypes.c_float else (i + 1) * (2 ** 33 if t is ctypes.c_int64 else 3) for i, (_, t) in enumerate(desc._fields_)]
        d = desc.from_buffer_copy(pack(*values))
        assert [getattr(d, n) for n, _ in desc._fields_] == values


def test_attend_refuses_more_threads_than_a_launch_takes(L):
    """2^32 threads and more in one direction: a refusal, not the runtime's error."""
    one = kvd(n_kv_heads=1)
    full = L.stq_kv_bytes(ctypes.byref(one))
    for kw in (dict(n_heads=1, q_stride=128, o_stride=128), dict(n_heads=65, q_stride=65 * 128, o_stride=65 * 128)):
        a = ad(n_req=1 << 24, **kw)
        assert L.stq_kv_attend(ctypes.byref(one), D, full, ctypes.byref(a), D, D, D, D, P(0x20000), None, 0, None) == -5, kw


def _import_alone(tmp_path, code, keep=("libstq.so",)):
    """Runs `code` where the package has its sources and the files of `keep` only."""
    import os
    import shutil
    import subprocess
    import sys
    import quantized_linear_attention_amd as q
    src = os.path.dirname(q.library_path())
    pkg = tmp_path / os.path.basename(src)
    pkg.mkdir()
    for f in os.listdir(src):
        if f.endswith(".py"):
            shutil.copy(os.path.join(src, f), pkg / f)
        elif f in keep:
            os.symlink(os.path.join(src, f), pkg / f)
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=240,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert r.returncode == 0, r.stderr
    return r.stdout


ALLOCATE = """
import numpy as np, quantized_linear_attention_amd as stq
e = np.array([[4.0, 2.0, 1.0], [8.0, 1.0, 0.5]])
bits, obj = stq.stq_allocate_bits(e, np.array([1.0, 1.0]), 1, 12)
print(bits.tolist(), stq.stq_kv_bytes(10, 64, 2, 128))
"""


def test_import_without_the_compiled_checks(tmp_path):
    """The package's host side without _tensor.so: every check is Python's then."""
    want = _import_alone(tmp_path, ALLOCATE, ("libstq.so", "_tensor.so"))
    (tmp_path / "b").mkdir()
    assert _import_alone(tmp_path / "b", ALLOCATE) == want
    (tmp_path / "c").mkdir()
    _import_alone(tmp_path / "c", """
import torch, quantized_linear_attention_amd as stq
try:
    stq.make_kv(torch.zeros(1 << 20, dtype=torch.uint8), 64, 2, 128)
    raise SystemExit("taken")
except stq.StqError as e:
    assert "pages" in str(e)
x = torch.zeros(3, 2, 64)
try:
    stq.stq_qk_norm_rope(x, None, x, None)
    raise SystemExit("taken")
except stq.StqError as e:
    assert "q is on cpu" in str(e), e
""")


def test_import_with_checks_of_another_torch(tmp_path):
    """A _tensor.so that does not load, or that was compiled against another torch, is left aside."""
    want = _import_alone(tmp_path, ALLOCATE, ("libstq.so", "_tensor.so"))
    (tmp_path / "b").mkdir()
    assert _import_alone(tmp_path / "b", "open('quantized_linear_attention_amd/_tensor.so', 'w').write('no library')\n" + ALLOCATE) == want
    (tmp_path / "c").mkdir()
    code = "import torch\ntorch.__version__ = '1.0.0'\n" + ALLOCATE + "\nassert not hasattr(stq._lib._tensor, 'torch_version')\n"
    assert _import_alone(tmp_path / "c", code, ("libstq.so", "_tensor.so")) == want


def test_import_without_torch(tmp_path):
    want = _import_alone(tmp_path, ALLOCATE, ("libstq.so", "_tensor.so"))
    (tmp_path / "b").mkdir()
    assert _import_alone(tmp_path / "b", "import sys\nsys.modules['torch'] = None\n" + ALLOCATE, ("libstq.so", "_tensor.so")) == want


def test_binding_refuses_what_was_left_out(stq, monkeypatch):
    """None for any tensor that a call has to have is a StqError."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    b, i, l = torch.bfloat16, torch.int32, torch.int64
    kv = stq.make_kv(Fake([10 * 2 * 64 * 136], torch.uint8), 64, 2, 128)
    x, y = Fake([4, 2, 128], b), Fake([4, 2, 128], b, ptr=0x20000)
    calls = ((stq.stq_kv_plan, dict(cached=Fake([2], i), new=Fake([2], i), free=Fake([9], i), table=Fake([2, 5], i), block_tokens=48,
                                    n_blocks=10, tok_start=Fake([3], i), lens=Fake([2], i), pos=Fake([7], i), slots=Fake([7], l),
                                    used=Fake([1], i)), ("block_tokens", "n_blocks")),
             (stq.stq_kv_store, dict(kv=kv, slots=Fake([4], l), k=x, v=x), ("kv",)),
             (stq.stq_kv_fetch, dict(kv=kv, slots=Fake([4], l), k_out=x, v_out=y), ("kv",)),
             (stq.stq_kv_attend, dict(kv=kv, table=Fake([2, 5], i), tok_start=Fake([3], i), lens=Fake([2], i), q=x, o=y, scale=0.1,
                                      max_new=2, max_len=100), ("kv", "max_new", "max_len", "scale")),
             (stq.stq_qk_norm_rope, dict(q=x, k=x, q_out=y, k_out=y, pos=Fake([4], i), cos_sin=Fake([9, 64], torch.float32)), ("k",)))
    for call, args, skip in calls:
        for name in args:
            if name not in skip:
                with pytest.raises(stq.StqError):
                    call(**dict(args, **{name: None}), stream=0)
    with pytest.raises(stq.StqError):
        stq.make_kv(None, 64, 2, 128)


def test_calls_refuse_outputs_over_inputs(L):
    """Outputs that share bytes with an input, or with each other, and are not the input itself."""
    kv = kvd(n_kv_heads=2)
    full = L.stq_kv_bytes(ctypes.byref(kv))
    w = 4 * 128 * 2                                       # bytes of a token's four heads

    def attend(q, o, **kw):
        return L.stq_kv_attend(ctypes.byref(kv), D, full, ctypes.byref(ad(**kw)), D, D, D, P(q), P(o), None, 0, None)
    q = 0x100000
    for o, kw in ((q + 16, {}), (q - 16, {}), (q + w, {}), (q + 2 * w + 16, {}), (q, dict(o_stride=1024)), (q + w - 16, dict(q_stride=1024, o_stride=1024)),
                  (q + 3 * w + 16, dict(q_stride=1024, o_stride=1024)), (q + w, dict(q_stride=1024))):
        assert attend(q, o, **kw) == -1, (hex(o), kw)

    def norm(kw, q=0x100000, k=0x200000, qo=0x300000, ko=0x400000):
        return L.stq_qk_norm_rope(ctypes.byref(nd(**kw)), P(q), P(k), None, None, D, D, P(qo), P(ko), None)
    for kw, at in (({}, dict(qo=0x100010)), ({}, dict(qo=0x100000 - 16)), ({}, dict(ko=0x200000 + 512)), ({}, dict(ko=0x100000)),
                   ({}, dict(qo=0x200000)), ({}, dict(ko=0x300000 + 2 * w)), (dict(out_type=2, q_out_stride=512), dict(qo=0x100000)),
                   (dict(q_out_stride=520), dict(qo=0x100000)), (dict(n_tok=1), dict(qo=0x100000 + w - 16)),
                   (dict(out_type=2), dict(qo=0x100000 + 3 * w - 16))):
        assert norm(kw, **at) == -1, (kw, at)
