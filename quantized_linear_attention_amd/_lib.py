"""ctypes marshalling for libstq.so (no computation happens here); _tensor.so, where it is there, checks tensor arguments."""
import ctypes
import os
import struct

import numpy as np

try:
    import torch    # before the library: see _load
except ImportError:
    torch = None    # the host-only calls need none

_PKG = os.path.dirname(os.path.abspath(__file__))
_PATH = os.path.join(_PKG, "libstq.so")

STQ_OK = 0
STQ_GATE_HEAD, STQ_GATE_CHANNEL = 0, 1
STQ_UNIT_HEAD, STQ_UNIT_ROW = 0, 1
STQ_BF16, STQ_FP16, STQ_FP32 = 0, 1, 2
STQ_NORM_NONE, STQ_NORM_RMS, STQ_NORM_L2 = 0, 1, 2
STQ_ROT_HALVES, STQ_ROT_ADJACENT = 0, 1


class StqError(RuntimeError):
    def __init__(self, status, what):
        super().__init__("%s: %s" % (what, stq_status_str(status)))
        self.status = status


class _Desc(ctypes.Structure):
    _fields_ = [("n_slots", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("gate_kind", ctypes.c_int32), ("unit_kind", ctypes.c_int32),
                ("window", ctypes.c_int32), ("n_comp", ctypes.c_int32),
                ("unit_bits", ctypes.POINTER(ctypes.c_int32)),
                ("row_weight", ctypes.POINTER(ctypes.c_float))]


class _KvDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_blocks", "block_tokens", "n_kv_heads", "d")]


class _NormDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_tok", "n_q_heads", "n_k_heads", "d", "in_type", "out_type", "norm")] +
                [("eps", ctypes.c_float)] + [(n, ctypes.c_int32) for n in ("n_rot", "rot_pairs", "n_pos")] +
                [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")])


class _AttendDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_req", "n_tok", "n_heads", "type", "table_cols", "max_new", "max_len",
                                               "window", "n_sink")] +
                [("scale", ctypes.c_float)] + [(n, ctypes.c_int64) for n in ("q_stride", "o_stride")])


def _packer(desc):
    """The bytes of a descriptor from its fields' values (a call's host time is 0.4 us less than with a ctypes structure)."""
    f = struct.Struct("@" + "".join({ctypes.c_int32: "i", ctypes.c_float: "f", ctypes.c_int64: "q"}[t] for _, t in desc._fields_))
    assert f.size == ctypes.sizeof(desc)

    def pack(*values):
        try:
            return f.pack(*values)
        except (struct.error, OverflowError) as e:
            raise StqError(-1, "descriptor: %s" % e) from None
    return pack


_norm_desc, _attend_desc = _packer(_NormDesc), _packer(_AttendDesc)


def library_path():
    return _PATH


def _load():
    if not os.path.exists(_PATH):
        raise ImportError("libstq.so is not built (%s); run quantized_linear_attention_amd/build.py "
                          "or __graft_entry__.build()" % _PATH)
    # torch has been imported above: its HIP runtime then serves the library too.
    # Loaded the other way round there are two runtimes in the process, and the
    # library's sees no device.
    L = ctypes.CDLL(_PATH)
    P, I, St = ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p
    DP = ctypes.POINTER(_Desc)
    L.stq_status_str.restype = ctypes.c_char_p
    L.stq_status_str.argtypes = [I]
    L.stq_pool_bytes.restype = ctypes.c_size_t
    L.stq_pool_bytes.argtypes = [DP]
    L.stq_pool_create.restype = I
    L.stq_pool_create.argtypes = [DP, P, ctypes.c_size_t, St, ctypes.POINTER(P)]
    L.stq_pool_destroy.restype = I
    L.stq_pool_destroy.argtypes = [P]
    for name in ("stq_pool_store", "stq_pool_fetch"):
        getattr(L, name).restype = I
        getattr(L, name).argtypes = [P, P, I, P, St]
    L.stq_decode_step.restype = I
    L.stq_decode_step.argtypes = [P, P, I, P, P, P, P, P, P, St]
    L.stq_prefill.restype = I
    L.stq_prefill_states.restype = I
    L.stq_prefill_states.argtypes = [I, I, I, I, I, P, P, P, P, P, P, P, P, St]
    L.stq_decode_readout.restype = I
    L.stq_decode_readout.argtypes = [P, P, I, P, P, P, P, P, P, St]
    L.stq_decode_commit.restype = I
    L.stq_decode_commit.argtypes = [P, P, I, P, P, P, P, P, St]
    L.stq_allocate_bits.restype = I
    L.stq_allocate_bits.argtypes = [I, P, P, I, ctypes.c_double, P, P]
    L.stq_prefill.argtypes = [P, P, I, P, P, P, P, P, P, P, St]
    for name in ("stq_window_flush", "stq_requant_fixed_scales"):
        getattr(L, name).restype = I
        getattr(L, name).argtypes = [P, P, I, St]
    Z, I64 = ctypes.c_size_t, ctypes.c_int64
    KP, NP, AP = ctypes.POINTER(_KvDesc), P, P           # (a descriptor's bytes, or a reference to one)
    for name, args in (("stq_kv_plan", [I, P, P, P, I, I, I, P, I, I, P, P, P, P, P, St]),
                       ("stq_qk_norm_rope", [NP, P, P, P, P, P, P, P, P, St]),
                       ("stq_kv_store", [KP, P, Z, P, I, P, P, I64, I64, I, St]),
                       ("stq_kv_fetch", [KP, P, Z, P, I, P, P, I, St]),
                       ("stq_kv_attend", [KP, P, Z, AP, P, P, P, P, P, P, Z, St])):
        getattr(L, name).restype = I
        getattr(L, name).argtypes = args
    for name, args in (("stq_kv_bytes", [KP]), ("stq_kv_attend_bytes", [KP, AP])):
        getattr(L, name).restype = Z
        getattr(L, name).argtypes = args
    return L


_L = _load()


class _PythonChecks:
    """In the place of the compiled checks: they pass nothing, so every argument takes the steps in Python."""
    address = rows = staticmethod(lambda *a: None)


def _compiled_checks():
    """_tensor.so links against torch's C++ interface: it serves the torch that it was compiled with, and no other."""
    try:
        from . import _tensor as t
    except ImportError:
        return _PythonChecks
    return t if str(torch.__version__).split("+")[0] == t.torch_version else _PythonChecks


_tensor = _PythonChecks if torch is None else _compiled_checks()


def stq_status_str(status):
    return _L.stq_status_str(int(status)).decode()


def _check(status, what):
    if status != STQ_OK:
        raise StqError(status, what)


def make_desc(n_slots, n_heads, d_k, d_v, unit_bits, row_weight, gate_kind=STQ_GATE_HEAD,
              unit_kind=STQ_UNIT_HEAD, window=0, n_comp=0):
    """Build a stq_pool_desc; the returned object keeps its host arrays alive."""
    bits = np.ascontiguousarray(unit_bits, dtype=np.int32).reshape(-1)
    wt = np.ascontiguousarray(row_weight, dtype=np.float32).reshape(-1)
    d = _Desc(int(n_slots), int(n_heads), int(d_k), int(d_v), int(gate_kind), int(unit_kind),
              int(window), int(n_comp), bits.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
              wt.ctypes.data_as(ctypes.POINTER(ctypes.c_float)))
    d._keep = (bits, wt)
    return d


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(getattr(stream, "cuda_stream", stream))


def _dev(t, dtype, what, numel=None, device=None):
    """Device pointer of a contiguous CUDA tensor of `dtype`; with `numel`
    and `device`, also checks its element count and device, so that no kernel
    is handed a buffer shorter than the sizes it indexes."""
    if t is None:
        return None
    if not (t.is_cuda and t.is_contiguous() and t.dtype == dtype):
        raise StqError(-1, "%s must be a contiguous %s CUDA tensor" % (what, dtype))
    if numel is not None and t.numel() != numel:
        raise StqError(-1, "%s has %d elements, expected %d" % (what, t.numel(), numel))
    if device is not None and t.device != device:
        raise StqError(-1, "%s is on %s, the pool buffer on %s" % (what, t.device, device))
    return ctypes.c_void_p(t.data_ptr())


def stq_pool_bytes(desc):
    return int(_L.stq_pool_bytes(ctypes.byref(desc)))


class _Pool:
    def __init__(self, handle, desc, buf):
        self.handle, self.desc, self.buf = handle, desc, buf
        self.H, self.dk, self.dv = int(desc.n_heads), int(desc.d_k), int(desc.d_v)
        self.gate, self.unit = int(desc.gate_kind), int(desc.unit_kind)
        self.device = buf.device

    def sizes(self, n):
        """Element counts of the per-token tensors of a call on n requests."""
        H, dk, dv = self.H, self.dk, self.dv
        return {"q": n * H * dk, "k": n * H * dk, "v": n * H * dv, "o": n * H * dv,
                "a": n * H * (dk if self.gate == STQ_GATE_CHANNEL else 1), "b": n * H,
                "S": n * H * dk * dv}

    def __del__(self):
        if getattr(self, "handle", None):
            _L.stq_pool_destroy(self.handle)
            self.handle = None


def stq_pool_create(desc, buf, stream=None):
    """buf: uint8 CUDA tensor of at least stq_pool_bytes(desc) bytes (256-aligned)."""
    import torch
    out = ctypes.c_void_p()
    p = _dev(buf, torch.uint8, "pool buffer")
    _check(_L.stq_pool_create(ctypes.byref(desc), p, buf.numel(), _stream(stream), ctypes.byref(out)),
           "stq_pool_create")
    return _Pool(out, desc, buf)


def stq_pool_destroy(pool):
    if pool.handle:
        _check(_L.stq_pool_destroy(pool.handle), "stq_pool_destroy")
        pool.handle = None


def _slots(slots, pool=None):
    import torch
    return _dev(slots, torch.int32, "slots", device=None if pool is None else pool.device), int(slots.numel())


def _token_args(pool, n, names, tensors):
    """Pointers of the per-token tensors of a call on n requests (or n tokens),
    each checked against the pool's sizes and device."""
    import torch
    want = pool.sizes(n)
    return [_dev(t, torch.float32, nm, want[nm], pool.device) for nm, t in zip(names, tensors)]


def stq_pool_store(pool, slots, S, stream=None):
    """S: fp32 [n][H][d_k][d_v] on the pool's device."""
    sp, n = _slots(slots, pool)
    _check(_L.stq_pool_store(pool.handle, sp, n, _token_args(pool, n, ["S"], [S])[0], _stream(stream)),
           "stq_pool_store")


def stq_pool_fetch(pool, slots, S_out, stream=None):
    sp, n = _slots(slots, pool)
    _check(_L.stq_pool_fetch(pool.handle, sp, n, _token_args(pool, n, ["S"], [S_out])[0], _stream(stream)),
           "stq_pool_fetch")


def stq_decode_step(pool, slots, q, k, v, a, b, o, stream=None):
    sp, n = _slots(slots, pool)
    ptrs = _token_args(pool, n, "qkvabo", (q, k, v, a, b, o))
    _check(_L.stq_decode_step(pool.handle, sp, n, *ptrs, _stream(stream)), "stq_decode_step")


def _prompt_tokens(pool_or_dims, n, seq_start, q):
    """Token count of a packed prompt batch, from q's size, and the checks that
    need the start offsets: n + 1 entries, the last within the batch.  Reading
    the last offset copies one int32 from the device (a synchronisation of
    the current stream); the prefill is not on the per-token path."""
    import torch
    H, dk = pool_or_dims
    if seq_start is None or seq_start.numel() != n + 1:
        raise StqError(-1, "seq_start must have n + 1 = %d entries" % (n + 1))
    if q is None or q.numel() % (H * dk):
        raise StqError(-1, "q must be [tokens][H][d_k]")
    tok = q.numel() // (H * dk)
    _dev(seq_start, torch.int32, "seq_start", n + 1, q.device)
    last = int(seq_start[-1].item()) if n else 0
    if last > tok:
        raise StqError(-1, "seq_start[n] = %d exceeds the %d tokens of q" % (last, tok))
    return tok


def stq_prefill(pool, slots, seq_start, q, k, v, a, b, o, stream=None):
    import torch
    sp, n = _slots(slots, pool)
    tok = _prompt_tokens((pool.H, pool.dk), n, seq_start, q)
    ptrs = _token_args(pool, tok, "qkvabo", (q, k, v, a, b, o))
    _check(_L.stq_prefill(pool.handle, sp, n, _dev(seq_start, torch.int32, "seq_start"), *ptrs,
                          _stream(stream)),
           "stq_prefill")


def stq_allocate_bits(err, half_life, n_pivots, budget_bits):
    """Host numpy arrays: err [n][3] (4, 6, 8 bits), half_life [n]; returns (bits [n] int32, objective)."""
    import numpy as np
    e = np.ascontiguousarray(err, np.float64)
    hl = np.ascontiguousarray(half_life, np.float64)
    n = hl.size
    if e.shape != (n, 3):
        raise StqError(-1, "err must be [n][3]")
    bits = np.zeros(n, np.int32)
    obj = ctypes.c_double(0.0)
    _check(_L.stq_allocate_bits(n, e.ctypes.data_as(ctypes.c_void_p), hl.ctypes.data_as(ctypes.c_void_p),
                                int(n_pivots), float(budget_bits), bits.ctypes.data_as(ctypes.c_void_p),
                                ctypes.byref(obj)), "stq_allocate_bits")
    return bits, obj.value


class _Dims:
    """Sizes of a plain-state prefill, laid out as a pool's would be."""
    def __init__(self, H, dk, dv, gate, device):
        self.H, self.dk, self.dv, self.gate, self.device = H, dk, dv, gate, device

    sizes = _Pool.sizes


def stq_prefill_states(S, seq_start, q, k, v, a, b, o, gate_kind=STQ_GATE_HEAD, stream=None):
    """S: contiguous fp32 CUDA tensor [n][H][d_k][d_v], advanced in place."""
    import torch
    f = torch.float32
    if S is None or S.dim() != 4:
        raise StqError(-1, "S must be [n][H][d_k][d_v]")
    n, H, dk, dv = S.shape
    Sp = _dev(S, f, "S")
    dims = _Dims(H, dk, dv, int(gate_kind), S.device)
    tok = _prompt_tokens((H, dk), n, seq_start, q)
    ptrs = _token_args(dims, tok, "qkvabo", (q, k, v, a, b, o))
    _check(_L.stq_prefill_states(n, H, dk, dv, gate_kind, Sp, _dev(seq_start, torch.int32, "seq_start"), *ptrs,
                                 _stream(stream)),
           "stq_prefill_states")


def stq_decode_readout(pool, slots, q, k, v, a, b, o, stream=None):
    sp, n = _slots(slots, pool)
    ptrs = _token_args(pool, n, "qkvabo", (q, k, v, a, b, o))
    _check(_L.stq_decode_readout(pool.handle, sp, n, *ptrs, _stream(stream)), "stq_decode_readout")


def stq_decode_commit(pool, slots, q, k, v, a, b, stream=None):
    sp, n = _slots(slots, pool)
    ptrs = _token_args(pool, n, "qkvab", (q, k, v, a, b))
    _check(_L.stq_decode_commit(pool.handle, sp, n, *ptrs, _stream(stream)), "stq_decode_commit")


def stq_window_flush(pool, slots, stream=None):
    sp, n = _slots(slots, pool)
    _check(_L.stq_window_flush(pool.handle, sp, n, _stream(stream)), "stq_window_flush")


def stq_requant_fixed_scales(pool, slots, stream=None):
    sp, n = _slots(slots, pool)
    _check(_L.stq_requant_fixed_scales(pool.handle, sp, n, _stream(stream)), "stq_requant_fixed_scales")


# ------------------------------------------- the softmax layers' operators

_TYPES = {} if torch is None else {torch.bfloat16: STQ_BF16, torch.float16: STQ_FP16, torch.float32: STQ_FP32}


def _type(t, what, allowed=(STQ_BF16, STQ_FP16, STQ_FP32)):
    code = _TYPES.get(t.dtype)
    if code not in allowed:
        raise StqError(-1, "%s has element type %s" % (what, t.dtype))
    return code


def _ptr(t, dtype, what, numel, index):
    """Address of a contiguous CUDA tensor of `dtype` with `numel` elements on
    device `index`: one step of the compiled module (0.1 us, 0.3 in Python),
    and here what it did not pass, with the refusal's words."""
    p = _tensor.address(t, dtype, numel, index)
    if p is not None:
        return p
    if t is None:
        raise StqError(-1, "%s is missing" % what)
    p = _dev(t, dtype, what, numel)
    if t.get_device() != index:
        raise StqError(-1, "%s is on %s, expected cuda:%d" % (what, t.device, index))
    return p


def _heads(t, what, n, heads, d, index):
    """(address, token stride) of a [tokens][heads][d] CUDA tensor whose heads are
    contiguous within a token; n, heads, d, index: what it has to be (None: anything)."""
    r = _tensor.rows(t, n, heads, d, index)
    if r is not None:
        return r
    if t is None or t.dim() != 3:
        raise StqError(-1, "%s must be [tokens][heads][d]" % what)
    a, b, c = t.shape
    if (n is not None and a != n) or (heads is not None and b != heads) or (d is not None and c != d):
        raise StqError(-1, "%s is %s, expected [%s][%s][%s]" % (what, (a, b, c), n, heads, d))
    i = t.get_device()
    if i < 0 or (index is not None and i != index):
        raise StqError(-1, "%s is on %s, expected %s" % (what, t.device, "cuda" if index is None else "cuda:%d" % index))
    st, sh, sc = t.stride()
    if sc != 1 or (b > 1 and sh != c):
        raise StqError(-1, "%s: the heads of a token must be contiguous" % what)
    return t.data_ptr(), st if a > 1 else b * c     # one shorter than a token is the library's to refuse


def _there(**tensors):
    """Refuses arguments whose sizes a call reads but that were left out."""
    for what, t in tensors.items():
        if t is None:
            raise StqError(-1, "%s is missing" % what)


def _i32(*sizes):
    """Sizes that C takes in 32 bits (ctypes would drop the rest in silence)."""
    for x in sizes:
        if -2 ** 31 <= x < 2 ** 31:
            continue
        raise StqError(-1, "one of the sizes %s does not fit 32 bits" % (sizes,))


def _call(name, index, stream, *args):
    """One library call on device `index` and its current stream (or the given one)."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    else:
        stream = getattr(stream, "cuda_stream", stream)
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            r = getattr(_L, name)(*args, stream)
    else:
        r = getattr(_L, name)(*args, stream)
    if r != STQ_OK:
        raise StqError(r, name)


class _Kv:
    def __init__(self, desc, pages):
        self.desc, self.pages, self.index = desc, pages, pages.get_device()
        self.n_kv_heads, self.d = desc.n_kv_heads, desc.d
        self.ref, self.ptr, self.bytes = ctypes.byref(desc), pages.data_ptr(), pages.numel()


def stq_kv_bytes(n_blocks, block_tokens, n_kv_heads, d):
    """Bytes of the cache's device buffer; 0 for sizes the library does not take."""
    _i32(n_blocks, block_tokens, n_kv_heads, d)
    return _L.stq_kv_bytes(ctypes.byref(_KvDesc(n_blocks, block_tokens, n_kv_heads, d)))


def make_kv(pages, block_tokens, n_kv_heads, d):
    """The 4-bit key/value cache that lives in `pages`, a contiguous uint8 CUDA
    tensor: as many whole blocks as it holds.  No copy, no initialisation."""
    n = 0 if pages is None else pages.numel()
    _dev(pages, torch.uint8, "pages")
    _i32(block_tokens, n_kv_heads, d)
    desc = _KvDesc(1, block_tokens, n_kv_heads, d)
    one = _L.stq_kv_bytes(ctypes.byref(desc))
    if not one or n < one:
        raise StqError(-1, "pages of %d bytes hold no block of %s tokens, %s heads, d = %s" % (n, block_tokens, n_kv_heads, d))
    desc.n_blocks = min(n // one, 2 ** 31 - 1)
    return _Kv(desc, pages)


def stq_kv_plan(cached, new, free, table, block_tokens, n_blocks, tok_start, lens, pos, slots, used, stream=None):
    """cached, new int32 [n]; free int32; table int32 [n][cols], updated in place;
    outputs tok_start int32 [n+1], lens int32 [n], pos int32 [tokens], slots int64
    [tokens], used int32 [1]."""
    if table is None or pos is None or free is None:
        _there(table=table, pos=pos, free=free)
    i, dev = torch.int32, table.get_device()
    if table.dim() != 2:
        raise StqError(-1, "table must be [requests][columns]")
    n, cols = table.shape
    tok, nf = pos.numel(), free.numel()
    _i32(n, cols, tok, nf, n_blocks, block_tokens)
    _call("stq_kv_plan", dev, stream, n, _ptr(cached, i, "cached", n, dev), _ptr(new, i, "new", n, dev),
          _ptr(free, i, "free", nf, dev), nf, n_blocks,
          block_tokens, _ptr(table, i, "table", n * cols, dev), cols, tok,
          _ptr(tok_start, i, "tok_start", n + 1, dev), _ptr(lens, i, "lens", n, dev), _ptr(pos, i, "pos", tok, dev),
          _ptr(slots, torch.int64, "slots", tok, dev), _ptr(used, i, "used", 1, dev))


def stq_qk_norm_rope(q, k, q_out, k_out, norm=STQ_NORM_RMS, eps=1e-6, q_weight=None, k_weight=None, pos=None,
                     cos_sin=None, rot_pairs=STQ_ROT_HALVES, stream=None):
    """q, k [tokens][heads][d] (views with contiguous heads; k and k_out may be
    None); outputs of the same type or float32; weights float32 [d]; with a
    table cos_sin float32 [positions][n_rot], pos int32 [tokens]."""
    f = torch.float32
    qp, qs = _heads(q, "q", None, None, None, None)
    n, hq, d = q.shape
    dev = q.get_device()
    qop, qos = _heads(q_out, "q_out", n, hq, d, dev)
    ti, to = _type(q, "q"), _type(q_out, "q_out")
    kp, ks, kop, kos, hk = None, 0, None, 0, 0
    if k is not None:
        kp, ks = _heads(k, "k", n, None, d, dev)
        hk = k.shape[1]
        kop, kos = _heads(k_out, "k_out", n, hk, d, dev)
        if k.dtype is not q.dtype or k_out.dtype is not q_out.dtype:
            raise StqError(-1, "k and k_out must have the types of q and q_out")
    n_rot = n_pos = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2 or pos is None:
            raise StqError(-1, "a rotation takes cos_sin [positions][n_rot] and pos [tokens]")
        n_pos, n_rot = cos_sin.shape
        pos, cos_sin = _ptr(pos, torch.int32, "pos", n, dev), _ptr(cos_sin, f, "cos_sin", n_pos * n_rot, dev)
    elif pos is not None:
        raise StqError(-1, "pos without cos_sin")
    if q_weight is not None:
        q_weight = _ptr(q_weight, f, "q_weight", d, dev)
    if k_weight is not None:
        k_weight = _ptr(k_weight, f, "k_weight", d, dev)
    _i32(n, n_rot, n_pos, norm, rot_pairs)
    desc = _norm_desc(n, hq, hk, d, ti, to, norm, eps, n_rot, rot_pairs, n_pos, qs, ks, qos, kos)
    _call("stq_qk_norm_rope", dev, stream, desc, qp, kp, q_weight, k_weight, pos, cos_sin, qop, kop)


def stq_kv_store(kv, slots, k, v, stream=None):
    """slots int64 [tokens]; k, v [tokens][n_kv_heads][d] of one element type."""
    if slots is None:
        _there(slots=slots)
    n, dev = slots.numel(), kv.index
    _i32(n)
    kp, ks = _heads(k, "k", n, kv.n_kv_heads, kv.d, dev)
    vp, vs = _heads(v, "v", n, kv.n_kv_heads, kv.d, dev)
    if v.dtype is not k.dtype:
        raise StqError(-1, "k and v must have one element type")
    _call("stq_kv_store", dev, stream, kv.ref, kv.ptr, kv.bytes, _ptr(slots, torch.int64, "slots", n, dev), n,
          kp, vp, ks, vs, _type(k, "k"))


def stq_kv_fetch(kv, slots, k_out, v_out, stream=None):
    """slots int64 [tokens]; k_out, v_out contiguous [tokens][n_kv_heads][d] of one element type."""
    if slots is None or k_out is None:
        _there(slots=slots, k_out=k_out)
    n, dev = slots.numel(), kv.index
    _i32(n)
    want, ty = n * kv.n_kv_heads * kv.d, k_out.dtype
    _call("stq_kv_fetch", dev, stream, kv.ref, kv.ptr, kv.bytes, _ptr(slots, torch.int64, "slots", n, dev), n,
          _ptr(k_out, ty, "k_out", want, dev), _ptr(v_out, ty, "v_out", want, dev), _type(k_out, "k_out"))


def stq_kv_attend_bytes(kv, n_req, n_tok, n_heads, max_new, max_len, window=0, n_sink=0):
    """Bytes of the workspace that stq_kv_attend takes for these sizes (0: none)."""
    _i32(n_req, n_tok, n_heads, max_new, max_len, window, n_sink)
    return _L.stq_kv_attend_bytes(kv.ref, _attend_desc(n_req, n_tok, n_heads, STQ_BF16, 1, max_new, max_len, window, n_sink,
                                                       1.0, 0, 0))


def stq_kv_attend(kv, table, tok_start, lens, q, o, scale, max_new, max_len, window=0, n_sink=0, work=None, stream=None):
    """table int32 [requests][cols]; tok_start int32 [requests + 1]; lens int32
    [requests]; q, o [tokens][n_heads][d], bfloat16 or float16; work: uint8
    tensor of at least stq_kv_attend_bytes(...) bytes (None where that is 0)."""
    i, dev = torch.int32, kv.index
    if table is None or table.dim() != 2:
        raise StqError(-1, "table must be [requests][columns]")
    n, cols = table.shape
    qp, qs = _heads(q, "q", None, None, kv.d, dev)
    tok, heads, d = q.shape
    op, os_ = _heads(o, "o", tok, heads, d, dev)
    ty = _type(q, "q", (STQ_BF16, STQ_FP16))
    if o.dtype is not q.dtype:
        raise StqError(-1, "o must have the type of q")
    wp = wn = 0
    if work is not None:
        wn = work.numel()
        wp = _ptr(work, torch.uint8, "work", wn, dev)
    _i32(tok, cols, max_new, max_len, window, n_sink)
    desc = _attend_desc(n, tok, heads, ty, cols, max_new, max_len, window, n_sink, scale, qs, os_)
    _call("stq_kv_attend", dev, stream, kv.ref, kv.ptr, kv.bytes, desc, _ptr(table, i, "table", n * cols, dev),
          _ptr(tok_start, i, "tok_start", n + 1, dev), _ptr(lens, i, "lens", n, dev), qp, op, wp, wn)
