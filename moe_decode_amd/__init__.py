"""Python binding of libmoe_decode (ctypes; argument marshalling only).

Every computation runs in the HIP library.  PyTorch supplies device memory
and the current stream; this module only packs descriptors, allocates
workspaces with torch, and turns error codes into exceptions.  There is no
fallback: if the library is missing, importing the binding's functions raises.

A call runs on the current stream, or on `stream`: then what it allocates is
that stream's memory, and the caller has other streams wait for it before they
read its outputs.
"""
import collections
import ctypes
import functools
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIBPATH = os.path.join(HERE, "libmoe_decode.so")

Q8_0, Q4_0, I8_ROW, I4_ROW, Q4_1, I2_ROW = 1, 2, 3, 4, 5, 6
TYPES = {"q8_0": Q8_0, "q4_0": Q4_0, "i8_row": I8_ROW, "i4_row": I4_ROW, "q4_1": Q4_1, "i2_row": I2_ROW}
ROW_TYPES = (I8_ROW, I4_ROW, I2_ROW)
ACTS = {"gelu_tanh": 0, "silu": 1}
X_F32, X_BF16 = 0, 1

STATUS = {0: "MD_OK", 1: "MD_ERR_INVALID_ARG", 2: "MD_ERR_SHAPE", 3: "MD_ERR_UNSUPPORTED",
          4: "MD_ERR_ALIGNMENT", 5: "MD_ERR_WORKSPACE", 6: "MD_ERR_HIP"}

EXPORTS = ("md_abi_version", "md_status_string", "md_last_error_detail", "md_row_bytes", "md_prepare_layout",
           "md_qgemv_workspace_size", "md_qgemv", "md_route_workspace_size", "md_moe_route_topk",
           "md_ffn_workspace_size", "md_ffn_forward", "md_moe_workspace_size", "md_moe_layer_forward",
           "md_moe_layer_forward_timed", "md_moe_layer_forward_residual", "md_add",
           "md_hbm_read_probe", "md_moe_experts_forward", "md_expert_cache_reset", "md_expert_cache_plan",
           "md_expert_cache_fill", "md_moe_cached_workspace_size", "md_moe_cached_forward",
           "md_moe_layer_forward_noalloc", "md_moe_layer_stage_relaunch",
           "md_i8_quantize", "md_i8_matmul", "md_i8_linear_workspace_size", "md_i8_linear",
           "md_kv_append", "md_kv_attention_workspace_size", "md_kv_attention", "md_kv_read_pages",
           "md_kv_copy_pages", "md_kv_pages_reset", "md_kv_pages_extend", "md_kv_pages_fork",
           "md_kv_pages_truncate", "md_kv_pages_compact",
           "md_kv_attention_masked_workspace_size", "md_kv_attention_masked", "md_kv_tree", "md_kv_tree_window", "md_qk_norm_rope",
           "md_moe_route_workspace_size", "md_moe_route", "md_moe_routed_workspace_size",
           "md_moe_layer_forward_routed", "md_token_logprobs_workspace_size", "md_token_logprobs")
STAGES = {"shared": 0, "router": 1, "select": 2, "gateup": 3, "down": 4, "combine": 5}


class MDError(RuntimeError):
    def __init__(self, status, detail):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{self.name}: {detail}")


class QMatrixDesc(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("row_scale", ctypes.c_void_p)]


class FFNDesc(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("gate", QMatrixDesc), ("up", QMatrixDesc), ("down", QMatrixDesc)]


class MoELayerDesc(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("F", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("act", ctypes.c_int32), ("type", ctypes.c_int32),
                ("gate_q", ctypes.c_void_p), ("up_q", ctypes.c_void_p), ("down_q", ctypes.c_void_p),
                ("gate_scale", ctypes.c_void_p), ("up_scale", ctypes.c_void_p), ("down_scale", ctypes.c_void_p),
                ("W_r", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("has_shared", ctypes.c_int32), ("shared", FFNDesc)]


_lib = None


def lib():
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBPATH):
            raise ImportError(f"{LIBPATH} is missing: build it with `python -m moe_decode_amd.build`")
        # torch first: its HIP runtime is then the one the library binds to
        # (two runtimes in one process would each see the device as busy)
        import torch  # noqa: F401
        L = ctypes.CDLL(LIBPATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        psz = ctypes.POINTER(ctypes.c_size_t)
        sig = {
            "md_abi_version": (i32, []),
            "md_status_string": (ctypes.c_char_p, [i32]),
            "md_last_error_detail": (ctypes.c_char_p, []),
            "md_row_bytes": (ctypes.c_int64, [i32, i32]),
            "md_prepare_layout": (i32, [i32, i32, i32, i32, vp, vp, vp]),
            "md_qgemv_workspace_size": (i32, [vp, i32, psz]),
            "md_qgemv": (i32, [vp, vp, i32, i32, vp, vp, sz, vp]),
            "md_route_workspace_size": (i32, [i32, i32, i32, i32, psz]),
            "md_moe_route_topk": (i32, [vp, i32, i32, vp, vp, i32, i32, vp, vp, vp, vp, sz, vp]),
            "md_ffn_workspace_size": (i32, [vp, i32, psz]),
            "md_ffn_forward": (i32, [vp, vp, i32, vp, vp, sz, vp]),
            "md_moe_workspace_size": (i32, [vp, i32, psz]),
            "md_moe_layer_forward": (i32, [vp, vp, i32, vp, vp, vp, vp, sz, vp]),
            "md_moe_layer_forward_timed": (i32, [vp, vp, i32, vp, vp, vp, vp, sz, vp, i32, vp, vp]),
            "md_moe_layer_forward_residual": (i32, [vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
            "md_add": (i32, [vp, vp, vp, ctypes.c_int64, vp]),
            "md_hbm_read_probe": (i32, [vp, ctypes.c_size_t, ctypes.c_uint32, vp, i32, vp]),
            "md_moe_experts_forward": (i32, [vp, vp, i32, vp, vp, vp, vp, sz, vp]),
            "md_expert_cache_reset": (i32, [vp]),
            "md_expert_cache_plan": (i32, [vp, vp, i32, vp, vp, vp, vp]),
            "md_expert_cache_fill": (i32, [vp, vp, vp, vp, i32, vp]),
            "md_moe_cached_workspace_size": (i32, [vp, vp, i32, psz]),
            "md_moe_cached_forward": (i32, [vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp, vp, vp]),
            "md_moe_layer_forward_noalloc": (i32, [vp, vp, i32, vp, vp, vp, vp]),
            "md_moe_layer_stage_relaunch": (i32, [vp, vp, i32, vp, vp, vp, vp, sz, vp, i32]),
            "md_i8_quantize": (i32, [vp, i32, i32, i32, vp, vp, vp]),
            "md_i8_matmul": (i32, [vp, vp, vp, i32, vp, vp, i32, vp]),
            "md_i8_linear_workspace_size": (i32, [vp, i32, psz]),
            "md_i8_linear": (i32, [vp, vp, i32, i32, vp, vp, i32, vp, sz, vp]),
            "md_kv_append": (i32, [vp, vp, vp, i64, vp, i64, i32, vp]),
            "md_kv_attention_workspace_size": (i32, [vp, vp, i32, i32, i32, i32, psz]),
            "md_kv_attention": (i32, [vp, vp, vp, i32, i32, i64, ctypes.c_float, i32, i32, vp, i32, i64, vp, sz, vp]),
            "md_kv_read_pages": (i32, [vp, vp, i32, vp, vp, i32, vp]),
            "md_kv_copy_pages": (i32, [vp, vp, vp, i32, vp]),
            "md_kv_pages_reset": (i32, [vp]),
            "md_kv_pages_extend": (i32, [vp, vp, i32, i32, i32, vp, vp, vp]),
            "md_kv_pages_fork": (i32, [vp, vp, i32, vp, i32]),
            "md_kv_pages_truncate": (i32, [vp, vp, i32, i32]),
            "md_kv_pages_compact": (i32, [vp, vp, i32, vp, i32, vp, vp, vp]),
            "md_kv_attention_masked_workspace_size": (i32, [vp, vp, i32, vp, i32, psz]),
            "md_kv_attention_masked": (i32, [vp, vp, vp, i32, i32, i64, ctypes.c_float, vp, vp, i32, i64, vp, sz, vp]),
            "md_kv_tree": (i32, [vp, vp, vp, i32, vp, vp]),
            "md_kv_tree_window": (i32, [vp, vp, i32, i32, vp, i32, vp, vp]),
            "md_qk_norm_rope": (i32, [vp, vp, i32, vp, i32, i64, vp, i32, i64, i32, vp, i64, vp, i64, i32, vp]),
            "md_moe_route_workspace_size": (i32, [i32, i32, i32, psz]),
            "md_moe_route": (i32, [vp, vp, i32, i32, i32, vp, vp, i32, vp, vp, vp, vp, sz, vp]),
            "md_moe_routed_workspace_size": (i32, [vp, i32, psz]),
            "md_moe_layer_forward_routed": (i32, [vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]),
            "md_token_logprobs_workspace_size": (i32, [i32, i32, i32, psz]),
            "md_token_logprobs": (i32, [vp, i32, i64, i32, i32, vp, i32, ctypes.c_float, i32, vp, vp, vp, vp, vp, sz,
                                        vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(rc):
    if rc != 0:
        raise MDError(rc, lib().md_last_error_detail().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _workspace(nbytes, device, workspace, stream=None):
    """The workspace of a call on `stream` (None: the current one).  One made
    here is released when the call returns, while its kernels still run, so it
    has to be of their stream's memory: what is made there next runs after them."""
    import torch
    if nbytes == 0:
        return None, 0
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    if stream is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        with torch.cuda.stream(stream):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, nbytes


def _result(stream, make, *args, **kw):
    """make(*args, **kw): an output of a call on `stream` (None: the current
    one), of that stream's memory like the workspace.  The caller has the stream
    that is current now wait for the call and reads the output there, so its
    memory is not given out again before what that stream holds when it is
    released."""
    if stream is None:
        return make(*args, **kw)
    import torch
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def row_bytes(type_, cols):
    return lib().md_row_bytes(TYPES.get(type_, type_), cols)


class DevQMatrix:
    """A quantized matrix (or a stack of `count` experts) resident on the GPU in
    the library's device layout."""

    def __init__(self, type_, rows, cols, q, row_scale=None, count=1):
        self.type = TYPES.get(type_, type_)
        self.rows, self.cols, self.count = rows, cols, count
        self.q, self.row_scale = q, row_scale

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if not name.startswith("_i8"):      # what _i8_desc has checked and packed
            object.__setattr__(self, "_i8", None)

    def desc(self, expert=0):
        rb = row_bytes(self.type, self.cols)
        off = expert * self.rows * rb
        sc = None if self.row_scale is None else self.row_scale.data_ptr() + 4 * expert * self.rows
        return QMatrixDesc(self.type, self.rows, self.cols, self.q.data_ptr() + off, sc)

    def expert(self, e):
        """The matrix of expert e of a stack, as a one-matrix view."""
        per = self.rows * row_bytes(self.type, self.cols)
        sc = None if self.row_scale is None else self.row_scale[e * self.rows:(e + 1) * self.rows]
        return DevQMatrix(self.type, self.rows, self.cols, self.q[e * per:(e + 1) * per], sc, 1)

    @property
    def nbytes(self):
        extra = 4 * self.rows * self.count if self.row_scale is not None else 0
        return self.rows * self.count * row_bytes(self.type, self.cols) + extra


def prepare_layout(type_, rows, cols, count, src, dst, stream=None):
    _check(lib().md_prepare_layout(TYPES.get(type_, type_), rows, cols, count, _ptr(src), _ptr(dst), _stream(stream)))


def qgemv_workspace_size(W, batch):
    d = W.desc()
    need = ctypes.c_size_t(0)
    _check(lib().md_qgemv_workspace_size(ctypes.byref(d), batch, ctypes.byref(need)))
    return need.value


def qgemv(W, x, y=None, workspace=None, stream=None):
    """y[b] = W x[b]; x (batch x cols) fp32 or bf16 tensor on the GPU."""
    import torch
    L = lib()
    d = W.desc()
    batch = x.shape[0] if x.dim() == 2 else 1
    xt = X_BF16 if x.dtype == torch.bfloat16 else X_F32
    if y is None:
        y = _result(stream, torch.empty, batch, W.rows, dtype=torch.float32, device=x.device)
    need = ctypes.c_size_t(0)
    _check(L.md_qgemv_workspace_size(ctypes.byref(d), batch, ctypes.byref(need)))
    ws, wsb = _workspace(need.value, x.device, workspace, stream)
    _check(L.md_qgemv(ctypes.byref(d), _ptr(x), xt, batch, _ptr(y), _ptr(ws), wsb, _stream(stream)))
    return y


def route_workspace_size(T, H, E, k):
    need = ctypes.c_size_t(0)
    _check(lib().md_route_workspace_size(T, H, E, k, ctypes.byref(need)))
    return need.value


def moe_route_topk(x, Wr, bias, k, idx=None, gates=None, logits=None, workspace=None, stream=None):
    import torch
    T, H = x.shape
    E = Wr.shape[0]
    dev = x.device
    idx = _result(stream, torch.empty, T, k, dtype=torch.int32, device=dev) if idx is None else idx
    gates = _result(stream, torch.empty, T, k, dtype=torch.float32, device=dev) if gates is None else gates
    ws, wsb = _workspace(route_workspace_size(T, H, E, k), dev, workspace, stream)
    _check(lib().md_moe_route_topk(_ptr(x), T, H, _ptr(Wr), _ptr(bias), E, k, _ptr(idx), _ptr(gates), _ptr(logits),
                                   _ptr(ws), wsb, _stream(stream)))
    return idx, gates


class FFN:
    def __init__(self, act, gate, up, down):
        self.act, self.gate, self.up, self.down = ACTS.get(act, act), gate, up, down

    def desc(self):
        return FFNDesc(self.act, self.gate.desc(), self.up.desc(), self.down.desc())


def ffn_workspace_size(ffn, T):
    d = ffn.desc()
    need = ctypes.c_size_t(0)
    _check(lib().md_ffn_workspace_size(ctypes.byref(d), T, ctypes.byref(need)))
    return need.value


def ffn_forward(ffn, x, y=None, workspace=None, stream=None):
    import torch
    T = x.shape[0]
    d = ffn.desc()
    if y is None:
        y = _result(stream, torch.empty, T, ffn.down.rows, dtype=torch.float32, device=x.device)
    ws, wsb = _workspace(ffn_workspace_size(ffn, T), x.device, workspace, stream)
    _check(lib().md_ffn_forward(ctypes.byref(d), _ptr(x), T, _ptr(y), _ptr(ws), wsb, _stream(stream)))
    return y


class MoELayer:
    """Device-resident MoE layer: gate/up/down are DevQMatrix stacks of E experts."""

    def __init__(self, H, F, E, k, act, gate, up, down, Wr, bias=None, shared=None):
        self.H, self.F, self.E, self.k = H, F, E, k
        self.act = ACTS.get(act, act)
        self.gate, self.up, self.down = gate, up, down
        self.Wr, self.bias, self.shared = Wr, bias, shared
        self._desc = None

    def desc(self):
        if self._desc is None:
            d = MoELayerDesc()
            d.H, d.F, d.E, d.k, d.act, d.type = self.H, self.F, self.E, self.k, self.act, self.gate.type
            d.gate_q, d.up_q, d.down_q = _ptr(self.gate.q), _ptr(self.up.q), _ptr(self.down.q)
            d.gate_scale, d.up_scale, d.down_scale = (_ptr(self.gate.row_scale), _ptr(self.up.row_scale),
                                                      _ptr(self.down.row_scale))
            d.W_r, d.router_bias = _ptr(self.Wr), _ptr(self.bias)
            d.has_shared = 1 if self.shared is not None else 0
            if self.shared is not None:
                d.shared = self.shared.desc()
            self._desc = d
        return self._desc

    def weight_bytes(self, n_experts_read):
        """Algorithmic weight bytes of one call that reads n_experts_read experts."""
        per = (self.gate.nbytes + self.up.nbytes + self.down.nbytes) // self.E
        b = n_experts_read * per + 4 * self.E * self.H + (4 * self.E if self.bias is not None else 0)
        if self.shared is not None:
            b += self.shared.gate.nbytes + self.shared.up.nbytes + self.shared.down.nbytes
        return b


def moe_workspace_size(layer, T, routed=False):
    """routed: of a call with a Routing."""
    d = layer.desc()
    need = ctypes.c_size_t(0)
    size = lib().md_moe_routed_workspace_size if routed else lib().md_moe_workspace_size
    _check(size(ctypes.byref(d), T, ctypes.byref(need)))
    return need.value


def moe_layer_forward(layer, x, y=None, idx=None, gates=None, workspace=None, stream=None, residual=None,
                      routing=None):
    """y = layer(x), or residual + layer(x) when a residual ([T][H] fp32,
    possibly x or y) is given.  routing (a Routing): in place of the layer's own
    top-k; a residual is then added by the caller (add)."""
    import torch
    T = x.shape[0]
    dev = x.device
    d = layer.desc()
    if routing is not None:
        if residual is not None:
            raise ValueError("a layer with a routing takes no residual")
        _dense("x", x, (T, layer.H), torch.float32, dev)
        with _on(dev, stream) as st:
            r = routing.desc(layer.E, dev)
            y = _result(stream, torch.empty, T, layer.H, dtype=torch.float32, device=dev) if y is None else \
                _dense("y", y, (T, layer.H), torch.float32, dev)
            if idx is not None:
                _dense("idx", idx, (T, layer.k), torch.int32, dev)
            if gates is not None:
                _dense("gates", gates, (T, layer.k), torch.float32, dev)
            ws, wsb = _workspace(moe_workspace_size(layer, T, True), dev, workspace, stream)
            _check(lib().md_moe_layer_forward_routed(ctypes.byref(d), r, _ptr(x), T, _ptr(y), _ptr(idx), _ptr(gates),
                                                     _ptr(ws), wsb, st))
        return y
    if y is None:
        y = _result(stream, torch.empty, T, layer.H, dtype=torch.float32, device=dev)
    ws, wsb = _workspace(moe_workspace_size(layer, T), dev, workspace, stream)
    if residual is None:
        _check(lib().md_moe_layer_forward(ctypes.byref(d), _ptr(x), T, _ptr(y), _ptr(idx), _ptr(gates), _ptr(ws), wsb,
                                          _stream(stream)))
    else:
        _check(lib().md_moe_layer_forward_residual(ctypes.byref(d), _ptr(x), T, _ptr(residual), _ptr(y), _ptr(idx),
                                                   _ptr(gates), _ptr(ws), wsb, _stream(stream)))
    return y


def moe_layer_stage_relaunch(layer, x, stage, y, workspace, idx=None, gates=None, stream=None):
    """Re-enqueue one stage ("shared", "router", "select", "gateup", "down",
    "combine") of an earlier moe_layer_forward made with the same x, y, idx,
    gates and workspace (a measurement aid)."""
    d = layer.desc()
    wsb = workspace.numel() * workspace.element_size()
    _check(lib().md_moe_layer_stage_relaunch(ctypes.byref(d), _ptr(x), x.shape[0], _ptr(y), _ptr(idx), _ptr(gates),
                                             _ptr(workspace), wsb, _stream(stream), STAGES.get(stage, stage)))


def moe_layer_forward_noalloc(layer, x, y, idx=None, gates=None, stream=None):
    """y = layer(x) with the library's built-in scratch (no workspace; the
    caller passes the output buffers).  Calls on one GPU must not overlap."""
    d = layer.desc()
    _check(lib().md_moe_layer_forward_noalloc(ctypes.byref(d), _ptr(x), x.shape[0], _ptr(y), _ptr(idx), _ptr(gates),
                                              _stream(stream)))
    return y


def moe_layer_forward_timed(layer, x, stage, start, stop, y=None, idx=None, gates=None, workspace=None,
                            stream=None):
    """moe_layer_forward that records the torch.cuda.Event pair start/stop
    around one stage ("shared", "router", "select", "gateup", "down",
    "combine") on the stream the kernels run on."""
    import torch
    T = x.shape[0]
    dev = x.device
    d = layer.desc()
    if y is None:
        y = _result(stream, torch.empty, T, layer.H, dtype=torch.float32, device=dev)
    ws, wsb = _workspace(moe_workspace_size(layer, T), dev, workspace, stream)
    _check(lib().md_moe_layer_forward_timed(ctypes.byref(d), _ptr(x), T, _ptr(y), _ptr(idx), _ptr(gates), _ptr(ws),
                                            wsb, _stream(stream), STAGES.get(stage, stage), start.cuda_event,
                                            stop.cuda_event))
    return y


def add(a, b, out=None, stream=None):
    """out = a + b (fp32 tensors of the same size on the device): the residual
    add between stacked layers."""
    import torch
    if out is None:
        out = _result(stream, torch.empty_like, a)
    _check(lib().md_add(_ptr(a), _ptr(b), _ptr(out), a.numel(), _stream(stream)))
    return out


def hbm_read_probe(src, sink, key=0xFFFFFFFF, workgroups=0, stream=None):
    """Reads every byte of the device tensor src once (a bandwidth
    measurement).  Nothing is written unless some lane's xor of the words it
    read equals key: for zeroed src, any nonzero key leaves sink (a device
    tensor of at least 4 bytes) untouched."""
    nbytes = src.numel() * src.element_size()
    _check(lib().md_hbm_read_probe(_ptr(src), nbytes, key, _ptr(sink), workgroups, _stream(stream)))


def moe_experts_forward(layer, x, idx, gates, y=None, workspace=None, stream=None):
    """The layer's experts for a given routing (idx int32, gates fp32, [T][k]
    on the device): y[t] = sum_j gates[t][j] * expert idx[t][j] (x[t])."""
    import torch
    T = x.shape[0]
    d = layer.desc()
    if y is None:
        y = _result(stream, torch.empty, T, layer.H, dtype=torch.float32, device=x.device)
    ws, wsb = _workspace(moe_workspace_size(layer, T), x.device, workspace, stream)
    _check(lib().md_moe_experts_forward(ctypes.byref(d), _ptr(x), T, _ptr(idx), _ptr(gates), _ptr(y), _ptr(ws), wsb,
                                        _stream(stream)))
    return y


class ExpertCacheState(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("S", ctypes.c_int32),
                ("slot_of_expert", ctypes.c_void_p), ("expert_in_slot", ctypes.c_void_p),
                ("uses", ctypes.c_void_p), ("last_use", ctypes.c_void_p), ("slot_idx", ctypes.c_void_p),
                ("step", ctypes.c_int64), ("hits", ctypes.c_int64), ("misses", ctypes.c_int64)]


class ExpertCache:
    """The replacement state of an S-slot expert cache over E experts (host
    arrays owned here, the policy in the library)."""

    def __init__(self, E, S):
        import numpy as np
        self.slot_of_expert = np.empty(E, dtype=np.int32)
        self.expert_in_slot = np.empty(S, dtype=np.int32)
        self.uses = np.empty(S, dtype=np.int64)
        self.last_use = np.empty(S, dtype=np.int64)
        self.slot_idx = np.empty(128 * 8, dtype=np.int32)
        self.state = ExpertCacheState(E, S, self.slot_of_expert.ctypes.data, self.expert_in_slot.ctypes.data,
                                      self.uses.ctypes.data, self.last_use.ctypes.data, self.slot_idx.ctypes.data,
                                      0, 0, 0)
        self.reset()

    def reset(self):
        _check(lib().md_expert_cache_reset(ctypes.byref(self.state)))

    def plan(self, idx):
        """One policy step for the expert ids idx (host int32): returns the slot
        ids and the (expert, slot) pairs to load."""
        import numpy as np
        idx = np.ascontiguousarray(idx, dtype=np.int32).reshape(-1)
        n = idx.size
        slots = np.empty(n, dtype=np.int32)
        me = np.empty(n, dtype=np.int32)
        ms = np.empty(n, dtype=np.int32)
        nm = ctypes.c_int32(0)
        _check(lib().md_expert_cache_plan(ctypes.byref(self.state), idx.ctypes.data, n, slots.ctypes.data,
                                          me.ctypes.data, ms.ctypes.data, ctypes.byref(nm)))
        return slots, list(zip(me[:nm.value].tolist(), ms[:nm.value].tolist()))

    @property
    def hits(self):
        return self.state.hits

    @property
    def misses(self):
        return self.state.misses


class ExpertTier:
    """A MoE layer whose experts live in (pinned) host memory, with S slots of
    HBM caching them: `host` is a MoELayer whose expert stacks are host
    tensors (router weights on the device); the slots are allocated here."""

    def __init__(self, host, S, device="cuda", shared=None, overlap=True):
        import torch
        self.host = host
        self.S = S
        # the misses load on a stream of their own while the shared expert runs
        self.copy_stream = torch.cuda.Stream(device=device) if overlap else None
        self.copy_done = torch.cuda.Event() if overlap else None
        if self.copy_done is not None:
            self.copy_done.record(self.copy_stream)   # torch creates the HIP event at its first record

        def slots_like(m, rows):
            q = torch.empty(S * rows * row_bytes(m.type, m.cols), dtype=torch.uint8, device=device)
            sc = None if m.row_scale is None else torch.empty(S * rows, dtype=torch.float32, device=device)
            return DevQMatrix(m.type, m.rows, m.cols, q, sc, S)
        self.slots = MoELayer(host.H, host.F, S, host.k, host.act, slots_like(host.gate, host.F),
                              slots_like(host.up, host.F), slots_like(host.down, host.H), host.Wr, host.bias,
                              shared if shared is not None else host.shared)
        self.cache = ExpertCache(host.E, S)

    def workspace_size(self, T):
        need = ctypes.c_size_t(0)
        _check(lib().md_moe_cached_workspace_size(ctypes.byref(self.host.desc()), ctypes.byref(self.slots.desc()), T,
                                                  ctypes.byref(need)))
        return need.value

    def forward(self, x, y=None, idx=None, gates=None, workspace=None, stream=None):
        """y = layer(x) through the cache (one synchronisation per call)."""
        import torch
        T = x.shape[0]
        if y is None:
            y = _result(stream, torch.empty, T, self.host.H, dtype=torch.float32, device=x.device)
        ws, wsb = _workspace(self.workspace_size(T), x.device, workspace, stream)
        cs = self.copy_stream.cuda_stream if self.copy_stream is not None else None
        ev = self.copy_done.cuda_event if self.copy_done is not None else None
        _check(lib().md_moe_cached_forward(ctypes.byref(self.host.desc()), ctypes.byref(self.slots.desc()),
                                           ctypes.byref(self.cache.state), _ptr(x), T, _ptr(y), _ptr(idx),
                                           _ptr(gates), _ptr(ws), wsb, _stream(stream), cs, ev))
        return y


# ---- the attention block in 8-bit integers -----------------------------------

_XTYPES = {}


def _xtype(dtype):
    t = _XTYPES.get(dtype)
    if t is None:
        import torch
        _XTYPES.update({torch.float32: X_F32, torch.bfloat16: X_BF16})
        if dtype not in _XTYPES:
            raise TypeError(f"float32 or bfloat16 wanted, got {dtype}")
        t = _XTYPES[dtype]
    return t


def _dense(name, t, shape, dtype, device):
    """Checks what the C call cannot see: a tensor's type, shape, layout, device."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on {device} wanted, got "
                         f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
    return t


def _rows(name, t, heads, dim, device):
    """A [rows][heads][dim] tensor whose rows may be strided (a slice of a
    projection's output): its row stride in values."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or t.device != device:
        raise ValueError(f"{name}: a tensor [rows][{heads}][{dim}] on {device} wanted, got {tuple(t.shape)} on "
                         f"{t.device}")
    st = t.stride()
    if shape[0] and ((dim > 1 and st[2] != 1) or (heads > 1 and st[1] != dim)):
        raise ValueError(f"{name}: a row's heads and channels must lie together, got strides {st}")
    return st[0] if shape[0] > 1 else heads * dim


def _raw_stream(index):
    """The handle of a device's current stream (its object costs 2 us to make,
    as long as a small kernel runs)."""
    global _raw_stream
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream(index)


def _current_device():
    """torch.cuda.current_device(), less its check that the GPU is initialised
    (the tensors are there)."""
    global _current_device
    import torch
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _current_device()


class _on:
    """The device of a call's tensors made current, and its stream's handle."""
    __slots__ = ("back", "stream")

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError(f"tensors on a GPU wanted, got {device}")
        now, want = _current_device(), device.index
        self.back = None
        if want is not None and want != now:
            import torch
            self.back = now
            torch.cuda.set_device(want)
            now = want
        self.stream = _raw_stream(now) if stream is None else stream.cuda_stream

    def __enter__(self):
        return self.stream

    def __exit__(self, *exc):
        if self.back is not None:
            import torch
            torch.cuda.set_device(self.back)


def _i8_desc(W, device=None):
    """The C descriptor of an int8 matrix, packed once while its attributes stay
    (DevQMatrix drops it when one is set); its tensors have to hold the matrix
    and lie on `device`."""
    q, r = W.q, W.row_scale
    made, at = W._i8, (q.data_ptr(), None if r is None else r.data_ptr())
    if made is None or made[0] != at:
        import torch
        if W.count != 1:
            raise ValueError(f"one matrix wanted, got a stack of {W.count}")
        if W.type == I8_ROW:
            if not q.is_contiguous() or q.nbytes < W.rows * W.cols:
                raise ValueError(f"W.q: {W.rows} x {W.cols} bytes wanted, got {tuple(q.shape)} of {q.dtype}, strides "
                                 f"{q.stride()}")
            if r is not None and (r.dtype != torch.float32 or not r.is_contiguous() or r.numel() < W.rows
                                  or r.device != q.device):
                raise ValueError(f"W.row_scale: {W.rows} float32 values on {q.device} wanted, got {tuple(r.shape)} of "
                                 f"{r.dtype} on {r.device}, strides {r.stride()}")
        made = W._i8 = (at, ctypes.byref(W.desc()), q.device)
    if device is not None and made[2] != device:
        raise ValueError(f"W is on {made[2]}, the call's tensors on {device}")
    return made[1]


def i8_quantize(x, codes=None, scales=None, stream=None):
    """The 8-bit codes of x ([T][K] fp32 or bf16) and their scale for each row."""
    import torch
    T, K = x.shape
    dev = x.device
    _dense("x", x, (T, K), x.dtype, dev)
    with _on(dev, stream) as st:
        codes = _result(stream, torch.empty, T, K, dtype=torch.int8, device=dev) if codes is None else \
            _dense("codes", codes, (T, K), torch.int8, dev)
        scales = _result(stream, torch.empty, T, dtype=torch.float32, device=dev) if scales is None else \
            _dense("scales", scales, (T,), torch.float32, dev)
        _check(lib().md_i8_quantize(_ptr(x), _xtype(x.dtype), T, K, _ptr(codes), _ptr(scales), st))
    return codes, scales


def _i8_args(W, T, bias, y, out_dtype, device, stream):
    import torch
    if bias is not None:
        _dense("bias", bias, (W.rows,), torch.float32, device)
    if y is None:
        return _result(stream, torch.empty, T, W.rows, dtype=out_dtype or torch.float32, device=device)
    if out_dtype is not None and y.dtype != out_dtype:
        raise ValueError(f"y is {y.dtype}, out_dtype {out_dtype}")
    return _dense("y", y, (T, W.rows), y.dtype, device)


def i8_matmul(W, codes, scales, bias=None, y=None, out_dtype=None, stream=None):
    """y[t][n] = scales[t] * W.row_scale[n] * sum_c codes[t][c] W[n][c] (+ bias[n])
    for an "i8_row" matrix W; y fp32 or bf16 (out_dtype, fp32 by default)."""
    import torch
    T, dev = codes.shape[0], codes.device
    _dense("codes", codes, (T, W.cols), torch.int8, dev)
    _dense("scales", scales, (T,), torch.float32, dev)
    with _on(dev, stream) as st:
        y = _i8_args(W, T, bias, y, out_dtype, dev, stream)
        _check(lib().md_i8_matmul(_i8_desc(W, dev), _ptr(codes), _ptr(scales), T, _ptr(bias), _ptr(y),
                                  _xtype(y.dtype), st))
    return y


def i8_linear_workspace_size(W, T):
    need = ctypes.c_size_t(0)
    _check(lib().md_i8_linear_workspace_size(_i8_desc(W), T, ctypes.byref(need)))
    return need.value


def i8_linear(W, x, bias=None, y=None, out_dtype=None, workspace=None, stream=None):
    """i8_matmul of i8_quantize(x): x [T][cols] fp32 or bf16, any T."""
    T, dev = x.shape[0], x.device
    _dense("x", x, (T, W.cols), x.dtype, dev)
    with _on(dev, stream) as st:
        y = _i8_args(W, T, bias, y, out_dtype, dev, stream)
        L, d = lib(), _i8_desc(W, dev)
        ws, wsb = None, 0
        if T > 1:
            made, key = W.__dict__.get("_i8_need"), (W.rows, W.cols, T)
            if made is None or made[0] != key:  # the last call's answer: the size follows from these alone
                made = W._i8_need = (key, i8_linear_workspace_size(W, T))
            ws, wsb = _workspace(made[1], dev, workspace, stream)
        _check(L.md_i8_linear(d, x.data_ptr(), _xtype(x.dtype), T, _ptr(bias), y.data_ptr(), _xtype(y.dtype), _ptr(ws),
                              wsb, st))
    return y


_I32_MAX = (1 << 31) - 1        # of a C int: ctypes passes the low 32 bits of what is larger


class KVMaskDesc(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("words", ctypes.c_int32),
                ("tree", ctypes.c_void_p)]


class KVCacheDesc(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class KVBatchDesc(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("rows", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("max_kv", ctypes.c_int32), ("table_stride", ctypes.c_int32), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p)]


class KVCache:
    """One layer's paged cache of keys and values in 8 bits: int8 codes
    k [n_pages][kv_heads][page][head_dim] and v [n_pages][kv_heads][head_dim][page],
    fp32 scales [n_pages][kv_heads]."""

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        if k.dim() != 4:
            raise ValueError(f"k: [n_pages][kv_heads][page][head_dim] wanted, got {tuple(k.shape)}")
        self.n_pages, self.kv_heads, self.page, self.head_dim = k.shape
        dev = self.device = k.device
        n, h, p, d = k.shape
        self.k = _dense("k", k, (n, h, p, d), torch.int8, dev)
        self.v = _dense("v", v, (n, h, d, p), torch.int8, dev)
        self.k_scale = _dense("k_scale", k_scale, (n, h), torch.float32, dev)
        self.v_scale = _dense("v_scale", v_scale, (n, h), torch.float32, dev)
        self.desc = KVCacheDesc(n, p, h, d, k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())
        self._ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, n_pages, kv_heads, head_dim, page=64, device="cuda"):
        import torch
        scale = lambda: torch.empty(n_pages, kv_heads, dtype=torch.float32, device=device)  # noqa: E731
        return cls(torch.empty(n_pages, kv_heads, page, head_dim, dtype=torch.int8, device=device),
                   torch.empty(n_pages, kv_heads, head_dim, page, dtype=torch.int8, device=device), scale(), scale())


class KVBatch:
    """Sequences with a run of new tokens each: q_start (int32 [S + 1]), kv_len
    (int32 [S]) and table (int32 [S][entries]) on the GPU, and the bounds max_q
    of the runs and max_kv of kv_len.  The arrays are read when the kernels run,
    so they may be rewritten in place between calls (and graph replays)."""

    def __init__(self, q_start, kv_len, table, max_q, max_kv):
        import torch
        S, dev = kv_len.shape[0], kv_len.device
        if table.dim() != 2:
            raise ValueError(f"table: [sequences][entries] wanted, got {tuple(table.shape)}")
        self.q_start = _dense("q_start", q_start, (S + 1,), torch.int32, dev)
        self.kv_len = _dense("kv_len", kv_len, (S,), torch.int32, dev)
        self.table = _dense("table", table, (S, table.shape[1]), torch.int32, dev)
        self.max_q, self.max_kv, self.device = max_q, max_kv, dev
        self._desc = KVBatchDesc(S, 0, max_q, max_kv, table.shape[1], q_start.data_ptr(), kv_len.data_ptr(),
                                 table.data_ptr())
        self._made, self._need = (-1, None), (None, 0)

    def desc(self, rows):
        """The C descriptor for a call on `rows` rows: the last one again, or a
        new one (one that another thread's call may be reading is not changed)."""
        made = self._made
        if made[0] != rows:
            d = KVBatchDesc.from_buffer_copy(self._desc)
            d.rows = rows
            made = self._made = (rows, ctypes.byref(d))
        return made[1]


def kv_append(cache, batch, k, v, stream=None):
    """Writes the rows of k and v ([rows][kv_heads][head_dim], fp32 or bf16, rows
    may be strided) into the cache as the batch's new tokens."""
    ks = _rows("k", k, cache.kv_heads, cache.head_dim, cache.device)
    vs = _rows("v", v, cache.kv_heads, cache.head_dim, cache.device)
    if k.dtype != v.dtype or k.shape[0] != v.shape[0] or batch.device != cache.device:
        raise ValueError(f"k and v of one type and length, the batch on {cache.device} wanted")
    with _on(cache.device, stream) as st:
        _check(lib().md_kv_append(cache._ref, batch.desc(k.shape[0]), _ptr(k), ks, _ptr(v),
                                  vs, _xtype(k.dtype), st))


def _mask_desc(causal, window, sinks, tree, rows, device):
    """What a call with a tree or sinks passes beside its window; None for a plain one."""
    if tree is None and not sinks:
        return None
    import torch
    if not causal:
        raise ValueError("a tree or sinks without causal")
    words = 0
    if tree is not None:
        words = tree.shape[1] if tree.dim() == 2 else 0
        _dense("tree", tree, (rows, words), torch.int64, device)
        if rows and not words:      # (its address is null, which the C call takes for no tree)
            raise ValueError("tree: masks of no words")
    return KVMaskDesc(window, sinks, words, _ptr(tree))


def kv_attention_workspace_size(cache, batch, rows, q_heads, causal=True, window=0, out_dtype=None, sinks=0, tree=None):
    import torch
    window, sinks = min(window, _I32_MAX), min(sinks, _I32_MAX)
    mask = _mask_desc(causal, window, sinks, tree, rows, cache.device)
    need, yt = ctypes.c_size_t(0), _xtype(out_dtype or torch.float32)
    if mask is None:
        _check(lib().md_kv_attention_workspace_size(cache._ref, batch.desc(rows), q_heads, int(causal), window, yt,
                                                    ctypes.byref(need)))
    else:
        _check(lib().md_kv_attention_masked_workspace_size(cache._ref, batch.desc(rows), q_heads, ctypes.byref(mask), yt,
                                                           ctypes.byref(need)))
    return need.value


def kv_attention(cache, batch, q, scale=None, causal=True, window=0, out=None, out_dtype=None, workspace=None,
                 stream=None, sinks=0, tree=None):
    """Attention of the batch's new rows q ([rows][q_heads][head_dim], fp32 or
    bf16, rows may be strided) over the cache; scale 1 / sqrt(head_dim) by
    default.  causal: a row sees the positions up to its own (window > 0: the
    last `window` of them, and with sinks the first `sinks` of the sequence);
    else every position of its sequence.  tree (int64 [rows][words], as kv_tree
    makes them): the run's tokens are the nodes of a tree, a row sees those whose
    bits are set, whatever the window, and the positions before the run (window
    > 0: the last of them, window less the tokens whose bits are set, and the
    first `sinks`); kv_tree with the same window and sinks sets no bit past them.
    out: fp32 or bf16 (out_dtype, fp32 by default); rows behind the last sequence
    are left as they are."""
    import torch
    if q.dim() != 3 or batch.device != cache.device:
        raise ValueError(f"q [rows][q_heads][head_dim] and the batch on {cache.device} wanted")
    rows, heads, dim = q.shape
    qs = _rows("q", q, heads, cache.head_dim, cache.device)
    window, sinks = min(window, _I32_MAX), min(sinks, _I32_MAX)     # more is as much
    mask = _mask_desc(causal, window, sinks, tree, rows, cache.device)
    with _on(cache.device, stream) as st:
        if out is None:
            out = _result(stream, torch.empty, rows, heads, dim, dtype=out_dtype or torch.float32,
                          device=cache.device)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
        if out.shape[0] != rows:
            raise ValueError(f"out has {out.shape[0]} rows, q {rows}")
        os_ = _rows("out", out, heads, cache.head_dim, cache.device)
        L, d, yt = lib(), batch.desc(rows), _xtype(out.dtype)
        key = (cache.page, cache.kv_heads, cache.head_dim, rows, heads, causal, window, yt)
        if mask is not None:
            key += (sinks, mask.words)
        made = batch._need  # the last call's answer: the size follows from these alone
        if made[0] != key:
            need = ctypes.c_size_t(0)
            if mask is None:
                _check(L.md_kv_attention_workspace_size(cache._ref, d, heads, int(causal), window, yt,
                                                        ctypes.byref(need)))
            else:
                _check(L.md_kv_attention_masked_workspace_size(cache._ref, d, heads, ctypes.byref(mask), yt,
                                                               ctypes.byref(need)))
            made = batch._need = (key, need.value)
        ws, wsb = _workspace(made[1], cache.device, workspace, stream)
        scale = dim ** -0.5 if scale is None else scale
        if mask is None:
            _check(L.md_kv_attention(cache._ref, d, _ptr(q), _xtype(q.dtype), heads, qs, scale, int(causal), window,
                                     _ptr(out), yt, os_, _ptr(ws), wsb, st))
        else:
            _check(L.md_kv_attention_masked(cache._ref, d, _ptr(q), _xtype(q.dtype), heads, qs, scale,
                                            ctypes.byref(mask), _ptr(out), yt, os_, _ptr(ws), wsb, st))
    return out


def kv_tree(batch, parents, masks=None, positions=None, stream=None, window=0, sinks=0):
    """The masks of the batch's trees of drafts, and their tokens' positions in
    the text, from each token's parent (int32 [rows] on the GPU: its number
    within the run, or -1).  window > 0 (with kv_attention's own): a token's mask
    has the last `window` tokens of its path, and those of it among the first
    `sinks` of the text.  Returns masks (int64 [rows][max_q / 64 rounded up], for
    kv_attention) and positions (int32 [rows], for qk_norm_rope)."""
    import torch
    rows, dev = parents.shape[0], batch.device
    window, sinks = min(window, _I32_MAX), min(sinks, _I32_MAX)
    _dense("parents", parents, (rows,), torch.int32, dev)
    with _on(dev, stream) as st:
        if masks is None:
            masks = _result(stream, torch.empty, rows, -(-batch.max_q // 64), dtype=torch.int64, device=dev)
        else:
            _dense("masks", masks, (rows, masks.shape[1]), torch.int64, dev)
        positions = _result(stream, torch.empty, rows, dtype=torch.int32, device=dev) if positions is None else \
            _dense("positions", positions, (rows,), torch.int32, dev)
        _check(lib().md_kv_tree_window(batch.desc(rows), _ptr(parents), window, sinks, _ptr(masks), masks.shape[1],
                                       _ptr(positions), st))
    return masks, positions


def kv_read_pages(cache, pages, k=None, v=None, out_dtype=None, stream=None):
    """The values that pages (int32 on the GPU) hold, keys and values both as
    [n][kv_heads][page][head_dim]."""
    import torch
    n, dev = pages.shape[0], cache.device
    _dense("pages", pages, (n,), torch.int32, dev)
    shape = (n, cache.kv_heads, cache.page, cache.head_dim)
    with _on(dev, stream) as st:
        dt = out_dtype or (k.dtype if k is not None else torch.float32)
        k = _result(stream, torch.empty, shape, dtype=dt, device=dev) if k is None else \
            _dense("k", k, shape, dt, dev)
        v = _result(stream, torch.empty, shape, dtype=dt, device=dev) if v is None else \
            _dense("v", v, shape, dt, dev)
        _check(lib().md_kv_read_pages(cache._ref, _ptr(pages), n, _ptr(k), _ptr(v), _xtype(dt), st))
    return k, v


def kv_copy_pages(cache, src, dst, stream=None):
    """Page dst[i] of the cache becomes page src[i] (host sequences of page
    numbers); a page that is written appears once among all of them."""
    from array import array
    src, dst = array("i", src), array("i", dst)
    n = len(src)
    if len(dst) != n:
        raise ValueError(f"{n} source pages and {len(dst)} destinations")
    with _on(cache.device, stream) as st:
        _check(lib().md_kv_copy_pages(cache._ref, src.buffer_info()[0], dst.buffer_info()[0], n, st))


class KVPagesState(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page", ctypes.c_int32), ("refs", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("n_free", ctypes.c_int32)]


class KVPages:
    """Which pages of a cache are in use (host state).  Sequences are kept here
    by a number each: their length and their row of `tables` (int32
    [max_seqs][entries], ready to be copied to the GPU)."""

    def __init__(self, n_pages, page, max_seqs, entries):
        import numpy as np
        self.refs, self.free = np.empty(n_pages, dtype=np.int32), np.empty(n_pages, dtype=np.int32)
        self._src, self._dst = np.empty(n_pages, dtype=np.int32), np.empty(n_pages, dtype=np.int32)
        self.tables = np.zeros((max_seqs, entries), dtype=np.int32)
        self.lens = np.zeros(max_seqs, dtype=np.int32)
        self.state = KVPagesState(n_pages, page, self.refs.ctypes.data, self.free.ctypes.data, 0)
        self.reset()

    def _row(self, s):
        if not 0 <= s < len(self.lens):
            raise IndexError(f"sequence {s} of {len(self.lens)}")
        return self.tables.ctypes.data + 4 * s * self.tables.shape[1]

    def reset(self):
        _check(lib().md_kv_pages_reset(ctypes.byref(self.state)))
        self.lens[:] = 0

    @property
    def n_free(self):
        return self.state.n_free

    def _pairs(self, n):
        return list(zip(self._src[:n].tolist(), self._dst[:n].tolist()))

    def extend(self, s, n_tokens):
        """Room for n_tokens more of sequence s: returns the (src, dst) page
        copies to make before they are appended (none, or one)."""
        n = ctypes.c_int32(0)
        new = int(self.lens[s]) + n_tokens
        _check(lib().md_kv_pages_extend(ctypes.byref(self.state), self._row(s), self.tables.shape[1],
                                        int(self.lens[s]), new, self._src.ctypes.data, self._dst.ctypes.data,
                                        ctypes.byref(n)))
        self.lens[s] = new
        return self._pairs(n.value)

    def fork(self, s, to, n_tokens=None):
        """Sequence `to` (an empty one) starts with s's first n_tokens (all)."""
        n = int(self.lens[s]) if n_tokens is None else n_tokens
        if s == to or not 0 <= n <= self.lens[s] or self.lens[to]:
            raise ValueError(f"fork {n} tokens of sequence {s} ({self.lens[s]}) into {to} ({self.lens[to]})")
        _check(lib().md_kv_pages_fork(ctypes.byref(self.state), self._row(s), n, self._row(to), self.tables.shape[1]))
        self.lens[to] = n

    def truncate(self, s, n_tokens=0):
        """Sequence s back to its first n_tokens."""
        _check(lib().md_kv_pages_truncate(ctypes.byref(self.state), self._row(s), int(self.lens[s]), n_tokens))
        self.lens[s] = n_tokens

    def compact(self):
        """Moves the used pages to the lowest numbers: the (src, dst) copies to
        make before the next use."""
        n = ctypes.c_int32(0)
        _check(lib().md_kv_pages_compact(ctypes.byref(self.state), self.tables.ctypes.data, self.tables.shape[1],
                                         self.lens.ctypes.data, len(self.lens), self._src.ctypes.data,
                                         self._dst.ctypes.data, ctypes.byref(n)))
        return self._pairs(n.value)


# ---- around the attention and the experts --------------------------------------

class RopeDesc(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inv_freq", ctypes.c_void_p), ("factor", ctypes.c_float), ("eps", ctypes.c_float),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p)]


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, factor=1.0,
                 q_out=None, k_out=None, out_dtype=None, stream=None):
    """The heads of q ([rows][q_heads][head_dim], fp32 or bf16, rows may be
    strided: a slice of a projection's output) and of k (likewise, or None) with
    their norms (over a head's channels, times weight fp32 [head_dim]; None: no
    norm), and their first 2 * len(inv_freq) channels turned by positions[row] *
    inv_freq (int32 [rows], fp32): channel p with p + len(inv_freq), interleaved:
    2 p with 2 p + 1; cosines and sines times factor.  q_out, k_out may be q and k
    themselves; out_dtype: the inputs' type by default.  Returns both."""
    import torch
    shape, dtype, dev = q.shape, q.dtype, q.device
    if len(shape) != 3:
        raise ValueError(f"q: [rows][heads][head_dim] wanted, got {tuple(shape)}")
    rows, heads, dim = shape
    qs, ks, kh = _rows("q", q, heads, dim, dev), 0, 0
    if k is not None:
        kshape = k.shape
        if len(kshape) != 3 or kshape[0] != rows or k.dtype is not dtype:
            raise ValueError(f"k: {rows} rows of {dtype} wanted, got {tuple(kshape)} of {k.dtype}")
        kh = kshape[1]
        ks = _rows("k", k, kh, dim, dev)
    _dense("positions", positions, (rows,), torch.int32, dev)
    half = inv_freq.numel()
    _dense("inv_freq", inv_freq, (half,), torch.float32, dev)
    qw = kw = None
    if q_weight is not None:
        qw = _dense("q_weight", q_weight, (dim,), torch.float32, dev).data_ptr()
    if k_weight is not None:
        kw = _dense("k_weight", k_weight, (dim,), torch.float32, dev).data_ptr()
    dt = out_dtype
    if dt is None:
        dt = q_out.dtype if q_out is not None else dtype if k_out is None else k_out.dtype

    def given(name, t, n):
        if t.dtype is not dt or t.shape[0] != rows:
            raise ValueError(f"{name}: {rows} rows of {dt} wanted, got {tuple(t.shape)} of {t.dtype}")
        return _rows(name, t, n, dim, dev)
    new = torch.empty if stream is None else functools.partial(_result, stream, torch.empty)
    with _on(dev, stream) as st:
        qo, ko, kp, kop = heads * dim, kh * dim, None, None
        if q_out is None:
            q_out = new(rows, heads, dim, dtype=dt, device=dev)
        else:
            qo = given("q_out", q_out, heads)
        if k is not None:
            if k_out is None:
                k_out = new(rows, kh, dim, dtype=dt, device=dev)
            else:
                ko = given("k_out", k_out, kh)
            kp, kop = k.data_ptr(), k_out.data_ptr()
        d = RopeDesc(dim, 2 * half, interleaved, inv_freq.data_ptr(), factor, eps, qw, kw)
        _check(lib().md_qk_norm_rope(ctypes.byref(d), positions.data_ptr(), rows, q.data_ptr(), heads, qs, kp, kh, ks,
                                     _xtype(dtype), q_out.data_ptr(), qo, kop, ko, _xtype(dt), st))
    return q_out, k_out if k is not None else None


SCORES = {"softmax": 0, "sigmoid": 1}


class RoutingDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_int32), ("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("groups_kept", ctypes.c_int32), ("best_two", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("scale", ctypes.c_float), ("balance", ctypes.c_void_p)]


class Routing:
    """How tokens are routed: k experts by "softmax" or "sigmoid" scores, chosen
    by score + balance (fp32 [E] on the GPU, or None) among the groups_kept best
    of `groups` equal runs of experts (by their largest, best_two: the sum of
    their two largest), with gates = scores (renorm: over their sum) times scale."""

    def __init__(self, k, score="softmax", balance=None, groups=1, groups_kept=1, best_two=False, renorm=True,
                 scale=1.0):
        self.k, self.score, self.balance = k, SCORES.get(score, score), balance
        self.groups, self.groups_kept, self.best_two = groups, groups_kept, bool(best_two)
        self.renorm, self.scale = bool(renorm), scale

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_made":         # what desc has checked and packed
            object.__setattr__(self, "_made", None)

    def desc(self, E, device):
        """The C descriptor for a call on E experts, packed once while the
        attributes stay."""
        b, made = self.balance, self._made
        at = None if b is None else b.data_ptr()
        if made is None or made[0] != at or made[1] != E or made[2] != device:
            import torch
            if b is not None:
                _dense("balance", b, (E,), torch.float32, device)
            d = RoutingDesc(self.k, self.score, self.groups, self.groups_kept, int(self.best_two), int(self.renorm),
                            self.scale, at)
            made = self._made = (at, E, device, ctypes.byref(d))
        return made[3]


def moe_route_workspace_size(T, H, E):
    need = ctypes.c_size_t(0)
    _check(lib().md_moe_route_workspace_size(T, H, E, ctypes.byref(need)))
    return need.value


@functools.lru_cache(maxsize=64)
def _route_need(device, T, H, E):
    """moe_route_workspace_size with `device` current: it follows from these alone."""
    return moe_route_workspace_size(T, H, E)


def moe_route(x, Wr, routing, bias=None, idx=None, gates=None, logits=None, workspace=None, stream=None):
    """The experts of each row of x ([T][H] fp32 or bf16, any T) and their gates
    ([T][k], int32 and fp32) for the router Wr ([E][H] fp32; bias fp32 [E], added
    to the logits): what moe_experts_forward takes, 128 tokens at a time."""
    import torch
    T, H = x.shape
    E, dev, dtype = Wr.shape[0], x.device, x.dtype
    _dense("x", x, (T, H), dtype, dev)
    _dense("Wr", Wr, (E, H), torch.float32, dev)
    if bias is not None:
        _dense("bias", bias, (E,), torch.float32, dev)
    if logits is not None:
        _dense("logits", logits, (T, E), torch.float32, dev)
    k = routing.k
    new = torch.empty if stream is None else functools.partial(_result, stream, torch.empty)
    with _on(dev, stream) as st:
        r = routing.desc(E, dev)
        idx = new(T, k, dtype=torch.int32, device=dev) if idx is None else \
            _dense("idx", idx, (T, k), torch.int32, dev)
        gates = new(T, k, dtype=torch.float32, device=dev) if gates is None else \
            _dense("gates", gates, (T, k), torch.float32, dev)
        ws, wsb = _workspace(_route_need(dev, T, H, E), dev, workspace, stream)
        _check(lib().md_moe_route(r, x.data_ptr(), _xtype(dtype), T, H, Wr.data_ptr(), _ptr(bias), E, idx.data_ptr(),
                                  gates.data_ptr(), _ptr(logits), _ptr(ws), wsb, st))
    return idx, gates


TokenLogprobs = collections.namedtuple("TokenLogprobs", "logprobs entropy top_ids top_logprobs")


def token_logprobs_workspace_size(rows, vocab, top=0):
    need = ctypes.c_size_t(0)
    _check(lib().md_token_logprobs_workspace_size(rows, vocab, top, ctypes.byref(need)))
    return need.value


@functools.lru_cache(maxsize=64)
def _logprobs_need(device, rows, vocab, top):
    """token_logprobs_workspace_size with `device` current: it follows from these alone."""
    return token_logprobs_workspace_size(rows, vocab, top)


def token_logprobs(logits, tokens=None, top=0, scale=1.0, logprobs=None, entropy=None, top_ids=None,
                   top_logprobs=None, workspace=None, stream=None):
    """From rows of logits ([rows][vocab] fp32 or bf16, rows may be strided),
    taken times scale (one over the temperature): the log probabilities of tokens
    (int32 [rows][n], None: none), the entropy, and the `top` largest logits' ids
    and log probabilities (None where top is 0)."""
    import torch
    shape, dev, dtype = logits.shape, logits.device, logits.dtype
    if len(shape) != 2:
        raise ValueError(f"logits: [rows][vocab] wanted, got {tuple(shape)}")
    rows, vocab = shape
    stride, one = logits.stride()
    if rows and vocab > 1 and one != 1:
        raise ValueError(f"logits: rows of neighbouring values wanted, got strides {(stride, one)}")
    f32, n, tok, lp = torch.float32, 0, None, None
    if tokens is not None:
        n = tokens.shape[1] if tokens.dim() == 2 else -1
        tok = _dense("tokens", tokens, (rows, n), torch.int32, dev).data_ptr()
    new = torch.empty if stream is None else functools.partial(_result, stream, torch.empty)
    with _on(dev, stream) as st:
        if tokens is not None:
            logprobs = new(rows, n, dtype=f32, device=dev) if logprobs is None else \
                _dense("logprobs", logprobs, (rows, n), f32, dev)
            lp = logprobs.data_ptr()
        entropy = new(rows, dtype=f32, device=dev) if entropy is None else \
            _dense("entropy", entropy, (rows,), f32, dev)
        ids = tlp = None
        if top:
            top_ids = new(rows, top, dtype=torch.int32, device=dev) if top_ids is None else \
                _dense("top_ids", top_ids, (rows, top), torch.int32, dev)
            top_logprobs = new(rows, top, dtype=f32, device=dev) if top_logprobs is None else \
                _dense("top_logprobs", top_logprobs, (rows, top), f32, dev)
            ids, tlp = top_ids.data_ptr(), top_logprobs.data_ptr()
        ws, wsb = _workspace(_logprobs_need(dev, rows, vocab, top), dev, workspace, stream)
        _check(lib().md_token_logprobs(logits.data_ptr(), _xtype(dtype), stride if rows > 1 else vocab, rows, vocab, tok, n,
                                       scale, top, lp, entropy.data_ptr(), ids, tlp, _ptr(ws), wsb, st))
    return TokenLogprobs(logprobs if tokens is not None else None, entropy, top_ids if top else None,
                         top_logprobs if top else None)
