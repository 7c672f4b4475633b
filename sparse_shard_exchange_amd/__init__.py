"""Python binding of libpw.so, the C ABI of the sharded-dataflow hot path.

Argument marshalling only: every step of the path runs in the library's HIP
kernels. PyTorch supplies device memory (tensors, the plan workspace) and the
stream (``torch.cuda.current_stream()``). The names mirror ``include/pw.h``.

Importing this package loads ``libpw.so`` from this directory and fails
loudly if it is missing: there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes as C
import os

# torch first: libpw.so links libamdhip64.so.7, and torch ships its own copy
# of that runtime under the same soname. Loaded after torch, our dependency
# resolves to torch's copy; loaded before, the process would end up with two
# HIP runtimes, and ours would find no device once torch's had claimed it.
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpw.so")

# ---- constants (include/pw.h) ------------------------------------------------
PW_ABI_VERSION = 1
PW_OK, PW_ERR_INVALID, PW_ERR_NOMEM, PW_ERR_DEVICE = 0, -1, -2, -3
PW_ERR_TIMEOUT, PW_ERR_BAD_DEST, PW_ERR_STATE, PW_ERR_UNSUPPORTED = -4, -5, -6, -7
PW_F32, PW_BF16 = 0, 1
PW_GRAPH_EXCHANGE, PW_GRAPH_CHAIN, PW_GRAPH_MOE, PW_GRAPH_PIPELINE = 0, 1, 2, 3
PW_OP_IDENTITY, PW_OP_AFFINE, PW_OP_ROWSUM = 0, 1, 2
PW_CHAIN_CHAINED, PW_CHAIN_OPBYOP, PW_CHAIN_FUSED, PW_CHAIN_SPLIT = 0, 1, 2, 3
PW_FLAG_TRACE, PW_FLAG_TIMING, PW_FLAG_STAGE_WINDOWS, PW_FLAG_ONE_LAUNCH = 0x1, 0x2, 0x4, 0x8
PW_NODE_ARG, PW_NODE_A, PW_NODE_EXCHANGE, PW_NODE_B, PW_NODE_RESULT, PW_NODE_STAGE = 0, 1, 2, 3, 4, 5


class pw_op(C.Structure):
    _fields_ = [("kind", C.c_uint32), ("a", C.c_float), ("b", C.c_float)]


class pw_plan_desc(C.Structure):
    _fields_ = [
        ("abi_version", C.c_uint32), ("kind", C.c_uint32), ("num_shards", C.c_uint32),
        ("num_src_shards", C.c_uint32), ("tuples_per_shard", C.c_uint64), ("payload_elems", C.c_uint32),
        ("dtype", C.c_uint32), ("a_op", pw_op), ("b_op", pw_op), ("top_k", C.c_uint32),
        ("hidden", C.c_uint32), ("microbatches", C.c_uint32), ("chain_mode", C.c_uint32),
        ("flags", C.c_uint32), ("capacity", C.c_uint32), ("spin_limit_ns", C.c_uint64),
        ("w_router", C.c_void_p), ("w1", C.c_void_p), ("w2", C.c_void_p),
    ]


class pw_sharded_buf(C.Structure):
    _fields_ = [
        ("base", C.c_void_p), ("num_tuples", C.c_uint64), ("num_shards", C.c_uint32),
        ("elems_per_tuple", C.c_uint32), ("dtype", C.c_uint32), ("reserved0", C.c_uint32),
        ("shard_offsets", C.c_void_p),
    ]


class pw_future_t(C.Structure):
    _fields_ = [("plan_id", C.c_uint64), ("node", C.c_uint32), ("shard", C.c_int32), ("epoch", C.c_uint64)]

    def __repr__(self):
        return f"pw_future_t(plan={self.plan_id}, node={self.node}, shard={self.shard}, epoch={self.epoch})"


class pw_exchange_io(C.Structure):
    _fields_ = [
        ("src", pw_sharded_buf), ("dest", C.c_void_p), ("dst", pw_sharded_buf), ("src_index", C.c_void_p),
        ("counts", C.c_void_p), ("b_out", C.c_void_p), ("result", C.c_void_p), ("logits", C.c_void_p),
        ("experts", C.c_void_p), ("gates", C.c_void_p),
    ]


class pw_kernel_time(C.Structure):
    _fields_ = [("name", C.c_char * 32), ("launches", C.c_uint64), ("total_ms", C.c_double)]


class pw_balance_desc(C.Structure):
    _fields_ = [("tokens", C.c_uint64), ("num_experts", C.c_uint32), ("top_k", C.c_uint32),
                ("balance_coef", C.c_float), ("z_coef", C.c_float)]


class pw_balance_io(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("logits", "experts", "valid", "counts", "prob_mean", "loss", "gates", "dgates",
                                          "grad_loss", "dlogits")]


class pw_moe_grad_desc(C.Structure):
    _fields_ = [("tokens", C.c_uint64), ("rows", C.c_uint64), ("d", C.c_uint32), ("num_experts", C.c_uint32),
                ("top_k", C.c_uint32), ("dtype", C.c_uint32)]


class pw_combine_grad_io(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("dout", "y", "gates", "src_index", "offsets", "valid", "dy", "dgates", "slot_of")]


class pw_dispatch_grad_io(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("dxd", "dlogits", "w_router", "x", "slot_of", "valid", "dx", "dw_router")]


class pw_norm_desc(C.Structure):
    _fields_ = [("rows", C.c_uint64), ("d", C.c_uint32), ("dtype", C.c_uint32), ("gates", C.c_uint32),
                ("x_scale", C.c_float), ("y_scale", C.c_float), ("eps", C.c_float)]


class pw_norm_io(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("x", "y", "w_y", "gate", "w_r", "r", "h", "dr", "dh", "valid", "dx", "dy", "dw_y",
                                          "dgate", "dw_r")]


PW_SCORE_SOFTMAX, PW_SCORE_SIGMOID = 0, 1


class pw_route_desc(C.Structure):
    _fields_ = [("tokens", C.c_uint64), ("num_experts", C.c_uint32), ("top_k", C.c_uint32), ("score", C.c_uint32),
                ("groups", C.c_uint32), ("top_groups", C.c_uint32), ("group_best", C.c_uint32), ("renorm", C.c_uint32),
                ("scale", C.c_float)]


class pw_route_io(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("logits", "bias", "valid", "experts", "weights", "dweights", "add", "dlogits")]


class pw_quant_desc(C.Structure):
    _fields_ = [("rows", C.c_uint64), ("d", C.c_uint32), ("dtype", C.c_uint32)]


class pw_quant_io(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("x", "limit", "q", "scale")]


class pw_q8_desc(C.Structure):
    _fields_ = [("rows", C.c_uint64), ("x_rows", C.c_uint64), ("d", C.c_uint32), ("n", C.c_uint32), ("num_experts", C.c_uint32),
                ("dtype", C.c_uint32), ("gather", C.c_uint32), ("scatter", C.c_uint32), ("gelu", C.c_uint32)]


class pw_q8_io(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("x", "q", "q_scale", "w", "w_scale", "offsets", "src_index", "out")]


class pw_combine_desc(C.Structure):
    _fields_ = [("tokens", C.c_uint64), ("d", C.c_uint32), ("top_k", C.c_uint32), ("dtype", C.c_uint32)]


class pw_topk_combine_io(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("y", "weights", "add", "out")]


PW_PROG_CHAIN, PW_PROG_EXCHANGE = 0, 1


class pw_store_stats(C.Structure):
    _fields_ = [
        ("base", C.c_uint64), ("capacity", C.c_uint64), ("in_use", C.c_uint64), ("pending_free", C.c_uint64),
        ("largest_free", C.c_uint64), ("objects", C.c_uint64), ("waiting", C.c_uint64), ("stalls", C.c_uint64),
        ("stalled_ms", C.c_double),
    ]


class pw_program(C.Structure):
    _fields_ = [
        ("kind", C.c_uint32), ("cost", C.c_uint32), ("plan", C.c_void_p), ("steps", C.c_uint64),
        ("state", pw_sharded_buf), ("aux", C.c_void_p), ("io", pw_exchange_io),
    ]


class pw_sched_record(C.Structure):
    _fields_ = [
        ("ticket", C.c_uint64), ("client", C.c_uint32), ("status", C.c_int32), ("dispatch", C.c_uint64),
        ("start_ms", C.c_double), ("end_ms", C.c_double),
    ]


# Every function the header declares, with its C signature.
_SIGNATURES = {
    "pw_abi_version": (C.c_uint32, []),
    "pw_strerror": (C.c_char_p, [C.c_int]),
    "pw_last_error": (C.c_char_p, []),
    "pw_plan": (C.c_int, [C.POINTER(pw_plan_desc), C.c_void_p, C.c_size_t, C.POINTER(C.c_size_t), C.POINTER(C.c_void_p)]),
    "pw_plan_destroy": (C.c_int, [C.c_void_p]),
    "pw_exchange": (C.c_int, [C.c_void_p, C.POINTER(pw_exchange_io), C.c_void_p, C.POINTER(pw_future_t)]),
    "pw_exchange_begin": (C.c_int, [C.c_void_p, C.POINTER(pw_exchange_io), C.c_void_p, C.c_void_p]),
    "pw_exchange_end": (C.c_int, [C.c_void_p, C.POINTER(pw_exchange_io), C.c_void_p, C.POINTER(pw_future_t)]),
    "pw_exchange_scratch": (C.c_int, [C.POINTER(pw_plan_desc), C.POINTER(pw_exchange_io), C.c_void_p]),
    "pw_chain_run": (C.c_int, [C.c_void_p, C.c_uint64, C.POINTER(pw_sharded_buf), C.c_void_p, C.c_void_p,
                               C.POINTER(pw_future_t)]),
    "pw_future_wait": (C.c_int, [pw_future_t, C.c_int64]),
    "pw_future_query": (C.c_int, [pw_future_t, C.POINTER(C.c_int)]),
    "pw_plan_read_futures": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t,
                                       C.POINTER(C.c_uint32), C.POINTER(C.c_uint32)]),
    "pw_plan_chain_placement": (C.c_int, [C.c_void_p, C.c_void_p, C.c_size_t]),
    "pw_plan_kernel_times": (C.c_int, [C.c_void_p, C.POINTER(pw_kernel_time), C.c_int, C.POINTER(C.c_int)]),
    "pw_plan_reset_times": (C.c_int, [C.c_void_p]),
    "pw_router_balance_workspace": (C.c_int, [C.POINTER(pw_balance_desc), C.POINTER(C.c_size_t)]),
    "pw_router_balance": (C.c_int, [C.POINTER(pw_balance_desc), C.POINTER(pw_balance_io), C.c_void_p, C.c_size_t,
                                    C.c_void_p]),
    "pw_router_grad": (C.c_int, [C.POINTER(pw_balance_desc), C.POINTER(pw_balance_io), C.c_void_p]),
    "pw_moe_combine_grad": (C.c_int, [C.POINTER(pw_moe_grad_desc), C.POINTER(pw_combine_grad_io), C.c_void_p]),
    "pw_moe_dispatch_grad_workspace": (C.c_int, [C.POINTER(pw_moe_grad_desc), C.POINTER(C.c_size_t)]),
    "pw_moe_dispatch_grad": (C.c_int, [C.POINTER(pw_moe_grad_desc), C.POINTER(pw_dispatch_grad_io), C.c_void_p,
                                       C.c_size_t, C.c_void_p]),
    "pw_block_norm": (C.c_int, [C.POINTER(pw_norm_desc), C.POINTER(pw_norm_io), C.c_void_p]),
    "pw_block_norm_grad_workspace": (C.c_int, [C.POINTER(pw_norm_desc), C.POINTER(C.c_size_t)]),
    "pw_block_norm_grad": (C.c_int, [C.POINTER(pw_norm_desc), C.POINTER(pw_norm_io), C.c_void_p, C.c_size_t,
                                     C.c_void_p]),
    "pw_route": (C.c_int, [C.POINTER(pw_route_desc), C.POINTER(pw_route_io), C.c_void_p]),
    "pw_route_grad": (C.c_int, [C.POINTER(pw_route_desc), C.POINTER(pw_route_io), C.c_void_p]),
    "pw_quant_rows": (C.c_int, [C.POINTER(pw_quant_desc), C.POINTER(pw_quant_io), C.c_void_p]),
    "pw_q8_product_workspace": (C.c_int, [C.POINTER(pw_q8_desc), C.POINTER(C.c_size_t)]),
    "pw_q8_product": (C.c_int, [C.POINTER(pw_q8_desc), C.POINTER(pw_q8_io), C.c_void_p, C.c_size_t, C.c_void_p]),
    "pw_topk_combine": (C.c_int, [C.POINTER(pw_combine_desc), C.POINTER(pw_topk_combine_io), C.c_void_p]),
    "pw_sched_create": (C.c_int, [C.c_uint32, C.POINTER(C.c_void_p)]),
    "pw_sched_add_client": (C.c_int, [C.c_void_p, C.c_uint32, C.POINTER(C.c_uint32)]),
    "pw_sched_submit": (C.c_int, [C.c_void_p, C.c_uint32, C.POINTER(pw_program), C.POINTER(C.c_uint64)]),
    "pw_sched_wait": (C.c_int, [C.c_void_p, C.c_uint64, C.c_int64]),
    "pw_sched_hold": (C.c_int, [C.c_void_p, C.c_int]),
    "pw_sched_records": (C.c_int, [C.c_void_p, C.POINTER(pw_sched_record), C.c_size_t, C.POINTER(C.c_size_t)]),
    "pw_sched_destroy": (C.c_int, [C.c_void_p]),
    "pw_store_create": (C.c_int, [C.c_size_t, C.POINTER(C.c_void_p)]),
    "pw_store_alloc": (C.c_int, [C.c_void_p, C.c_size_t, C.c_uint32, C.c_int64, C.POINTER(C.c_uint64),
                                 C.POINTER(C.c_void_p)]),
    "pw_store_free": (C.c_int, [C.c_void_p, C.c_uint64, C.c_void_p]),
    "pw_store_release_owner": (C.c_int, [C.c_void_p, C.c_uint32, C.c_void_p, C.POINTER(C.c_uint64)]),
    "pw_store_get_stats": (C.c_int, [C.c_void_p, C.POINTER(pw_store_stats)]),
    "pw_store_destroy": (C.c_int, [C.c_void_p]),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m sparse_shard_exchange_amd.build` "
                          "(the HIP library is the only implementation; there is no fallback)")
    lib = C.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.pw_abi_version() != PW_ABI_VERSION:
        raise ImportError(f"libpw ABI {lib.pw_abi_version()} != {PW_ABI_VERSION}")
    return lib


lib = _load()


class PwError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{lib.pw_strerror(code).decode()} ({code}): {msg}")
        self.code = code


def check(rc: int) -> int:
    if rc != PW_OK:
        raise PwError(rc, lib.pw_last_error().decode())
    return rc


def op(kind=PW_OP_IDENTITY, a=0.0, b=0.0) -> pw_op:
    return pw_op(kind, a, b)


def desc(kind, num_shards, tuples_per_shard, payload_elems=0, dtype=PW_F32, num_src_shards=0,
         a_op=None, b_op=None, top_k=0, hidden=0, microbatches=0, chain_mode=PW_CHAIN_CHAINED,
         flags=0, spin_limit_ns=0, w_router=None, w1=None, w2=None, capacity=0) -> pw_plan_desc:
    d = pw_plan_desc()
    d.abi_version = PW_ABI_VERSION
    d.kind = kind
    d.num_shards = num_shards
    d.num_src_shards = num_src_shards
    d.tuples_per_shard = tuples_per_shard
    d.payload_elems = payload_elems
    d.dtype = dtype
    d.a_op = a_op or op()
    d.b_op = b_op or op()
    d.top_k = top_k
    d.hidden = hidden
    d.microbatches = microbatches
    d.chain_mode = chain_mode
    d.flags = flags
    d.capacity = capacity
    d.spin_limit_ns = spin_limit_ns
    d.w_router = _ptr(w_router)
    d.w1 = _ptr(w1)
    d.w2 = _ptr(w2)
    return d


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def workspace_size(d: pw_plan_desc) -> int:
    """Host-only sizing call (no HIP)."""
    need = C.c_size_t(0)
    check(lib.pw_plan(C.byref(d), None, 0, C.byref(need), None))
    return need.value


def sharded(t, num_shards, elems_per_tuple, dtype, shard_offsets=None) -> pw_sharded_buf:
    b = pw_sharded_buf()
    b.base = _ptr(t)
    b.num_tuples = (t.numel() // elems_per_tuple) if (t is not None and elems_per_tuple) else 0
    b.num_shards = num_shards
    b.elems_per_tuple = elems_per_tuple
    b.dtype = dtype
    b.shard_offsets = _ptr(shard_offsets)
    return b


class Plan:
    """A built plan: the opaque handle plus the torch-allocated workspace it lives in."""

    def __init__(self, d: pw_plan_desc, device="cuda"):
        import torch
        self.desc = d
        self.ws_bytes = workspace_size(d)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=device)
        h = C.c_void_p()
        need = C.c_size_t(0)
        check(lib.pw_plan(C.byref(d), C.c_void_p(self.ws.data_ptr()), self.ws.numel(), C.byref(need), C.byref(h)))
        self.handle = h

    def destroy(self):
        if self.handle:
            check(lib.pw_plan_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            if getattr(self, "handle", None):
                lib.pw_plan_destroy(self.handle)
        except Exception:
            pass

    def exchange(self, io: pw_exchange_io, stream=None) -> pw_future_t:
        f = pw_future_t()
        check(lib.pw_exchange(self.handle, C.byref(io), _stream(stream), C.byref(f)))
        return f

    def exchange_begin(self, io: pw_exchange_io, num_dest: int, stream=None):
        """First half of a split step; blocks, returns the segment offsets
        (numpy int64 [num_dest + 1])."""
        import numpy as np
        offs = np.zeros(num_dest + 1, dtype=np.int64)
        check(lib.pw_exchange_begin(self.handle, C.byref(io), _stream(stream), C.c_void_p(offs.ctypes.data)))
        return offs

    def exchange_end(self, io: pw_exchange_io, stream=None) -> pw_future_t:
        f = pw_future_t()
        check(lib.pw_exchange_end(self.handle, C.byref(io), _stream(stream), C.byref(f)))
        return f

    def chain_run(self, steps: int, state: pw_sharded_buf, aux=None, stream=None) -> pw_future_t:
        f = pw_future_t()
        check(lib.pw_chain_run(self.handle, steps, C.byref(state), _ptr(aux), _stream(stream), C.byref(f)))
        return f

    def read_futures(self, trace=False):
        """(epochs, fires, stamps) as numpy arrays [nodes, width]."""
        import numpy as np
        nodes, width = C.c_uint32(0), C.c_uint32(0)
        check(lib.pw_plan_read_futures(self.handle, None, None, None, 0, C.byref(nodes), C.byref(width)))
        n = nodes.value * width.value
        ep = np.zeros(n, np.uint32)
        fi = np.zeros(n, np.uint32)
        st = np.zeros(n, np.uint64) if trace else None
        check(lib.pw_plan_read_futures(self.handle, ep.ctypes.data, fi.ctypes.data,
                                       st.ctypes.data if trace else None, n, C.byref(nodes), C.byref(width)))
        shape = (nodes.value, width.value)
        return ep.reshape(shape), fi.reshape(shape), (st.reshape(shape) if trace else None)

    def kernel_times(self) -> dict:
        n = C.c_int(0)
        check(lib.pw_plan_kernel_times(self.handle, None, 0, C.byref(n)))
        arr = (pw_kernel_time * max(n.value, 1))()
        check(lib.pw_plan_kernel_times(self.handle, arr, n.value, C.byref(n)))
        return {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms) for i in range(n.value)}

    def reset_times(self):
        check(lib.pw_plan_reset_times(self.handle))


def exchange_scratch(d: pw_plan_desc, io: pw_exchange_io, stream=None) -> None:
    """One EXCHANGE step with the library's static scratch tables (no plan,
    no workspace, nothing allocated); stream ordered, no future."""
    check(lib.pw_exchange_scratch(C.byref(d), C.byref(io), _stream(stream)))


def future_wait(f: pw_future_t, timeout_ns: int = -1) -> None:
    check(lib.pw_future_wait(f, timeout_ns))


def future_query(f: pw_future_t) -> bool:
    fired = C.c_int(0)
    check(lib.pw_future_query(f, C.byref(fired)))
    return bool(fired.value)


def exchange_io(src, dest, dst, num_src, num_dest, elems, dtype=PW_F32, src_index=None, counts=None,
                offsets=None, b_out=None, result=None, logits=None, experts=None, gates=None) -> pw_exchange_io:
    io = pw_exchange_io()
    io.src = sharded(src, num_src, elems, dtype)
    io.dest = _ptr(dest)
    io.dst = sharded(dst, num_dest, elems, dtype, offsets)
    io.src_index = _ptr(src_index)
    io.counts = _ptr(counts)
    io.b_out = _ptr(b_out)
    io.result = _ptr(result)
    io.logits = _ptr(logits)
    io.experts = _ptr(experts)
    io.gates = _ptr(gates)
    return io


class Exchange:
    """One EXCHANGE plan with its output buffers, for repeated steps on
    inputs of one shape. Allocation happens here, once; ``step`` only
    enqueues the library's kernels."""

    def __init__(self, num_shards, tuples_per_shard, payload_elems, dtype=PW_F32, num_src_shards=0,
                 a_op=None, b_op=None, flags=0, spin_limit_ns=0, want_index=True, want_counts=False,
                 device="cuda"):
        import torch
        self.N = num_shards
        self.S = num_src_shards or num_shards
        self.P = payload_elems
        self.dtype = dtype
        self.G = self.S * tuples_per_shard
        self.desc = desc(PW_GRAPH_EXCHANGE, num_shards, tuples_per_shard, payload_elems, dtype, num_src_shards,
                         a_op=a_op, b_op=b_op, flags=flags, spin_limit_ns=spin_limit_ns)
        self.plan = Plan(self.desc, device)
        tdt = torch.float32 if dtype == PW_F32 else torch.bfloat16
        self.dst = torch.empty((self.G, payload_elems), dtype=tdt, device=device)
        self.offsets = torch.empty(self.N + 1, dtype=torch.int64, device=device)
        self.src_index = torch.empty(self.G, dtype=torch.int32, device=device) if want_index else None
        self.counts = torch.empty((self.S, self.N), dtype=torch.int32, device=device) if want_counts else None
        bk = self.desc.b_op.kind
        if bk == PW_OP_ROWSUM:
            self.b_out = torch.empty(self.G, dtype=torch.float32, device=device)
        elif bk == PW_OP_AFFINE:
            self.b_out = torch.empty((self.G, payload_elems), dtype=torch.float32, device=device)
        else:
            self.b_out = None

    def io(self, x, dest) -> pw_exchange_io:
        return exchange_io(x, dest, self.dst, self.S, self.N, self.P, self.dtype, src_index=self.src_index,
                           counts=self.counts, offsets=self.offsets, b_out=self.b_out)

    def step(self, x, dest, stream=None) -> pw_future_t:
        return self.plan.exchange(self.io(x, dest), stream)


class Chain:
    """One CHAIN plan: N shards of E fp32, A and B elementwise, run in
    Chained, OpByOp or Fused mode."""

    def __init__(self, num_shards, elems, a_op=None, b_op=None, mode=PW_CHAIN_CHAINED, flags=0,
                 spin_limit_ns=0, device="cuda"):
        self.N, self.E = num_shards, elems
        self.desc = desc(PW_GRAPH_CHAIN, num_shards, elems, 0, PW_F32,
                         a_op=a_op or op(PW_OP_AFFINE, 1.0, 1.0), b_op=b_op or op(PW_OP_AFFINE, 0.5, 0.0),
                         chain_mode=mode, flags=flags, spin_limit_ns=spin_limit_ns)
        self.plan = Plan(self.desc, device)

    def run(self, state, steps, aux=None, stream=None) -> pw_future_t:
        return self.plan.chain_run(steps, sharded(state, self.N, self.E, PW_F32), aux, stream)

    def placement(self):
        """PW_CHAIN_SPLIT plans: numpy [N, 2] XCD of the waves that ran A[i], B[i]
        in the last call."""
        import numpy as np
        out = np.zeros(2 * self.N, np.uint32)
        check(lib.pw_plan_chain_placement(self.plan.handle, out.ctypes.data, out.size))
        return out.reshape(self.N, 2)


class Pipeline:
    """One PIPELINE plan: S stages of h = bf16(GELU(h . W_s)) over M microbatches
    of rows x d bf16, GPipe fill/drain, one launch per pass. W is [S][d][d]
    bf16, stored [in][out] (borrowed: keep it alive while the plan lives)."""

    def __init__(self, w, microbatches, rows, flags=0, spin_limit_ns=0, device="cuda"):
        import torch
        assert w.dtype == torch.bfloat16 and w.dim() == 3 and w.shape[1] == w.shape[2]
        self.w = w
        self.S, self.d = w.shape[0], w.shape[1]
        self.M, self.R = microbatches, rows
        self.desc = desc(PW_GRAPH_PIPELINE, self.S, rows, self.d, PW_BF16, microbatches=microbatches,
                         flags=flags, spin_limit_ns=spin_limit_ns, w1=w)
        self.plan = Plan(self.desc, device)

    def run(self, x, acts, stream=None) -> pw_future_t:
        """x: [M][rows][d] bf16; acts: [S][M][rows][d] bf16 receives every stage output."""
        return self.plan.chain_run(1, sharded(x, self.M, self.d, PW_BF16), acts, stream)


class MoE:
    """One MOE plan: router d x E + top-2 softmax gate, dispatch exchange to E
    expert shards, expert FFN d -> hidden -> d with GELU, gated combine.
    Weights (bf16, stored [in][out]) are borrowed: keep them alive."""

    def __init__(self, w_router, w1, w2, tokens, num_src_shards=64, flags=0, spin_limit_ns=0,
                 want_logits=True, want_counts=False, capacity=0, static_buffers=True, device="cuda"):
        import torch
        self.d, self.E = w_router.shape
        self.hidden = w1.shape[2]
        assert tokens % num_src_shards == 0
        self.T, self.S = tokens, num_src_shards
        self.w = (w_router, w1, w2)
        self.capacity = capacity
        self.device = device
        self.desc = desc(PW_GRAPH_MOE, self.E, tokens // num_src_shards, self.d, PW_BF16,
                         num_src_shards=num_src_shards, top_k=2, hidden=self.hidden, flags=flags,
                         spin_limit_ns=spin_limit_ns, w_router=w_router, w1=w1, w2=w2, capacity=capacity)
        self.plan = Plan(self.desc, device)
        bf = torch.bfloat16
        # dispatched rows at most: every tuple, or E * capacity if fewer
        self.static_rows = min(2 * tokens, self.E * capacity) if capacity else 2 * tokens
        rows = self.static_rows if static_buffers else 0  # split_step allocates them per step
        self.xd = torch.empty((rows, self.d), dtype=bf, device=device)
        self.y = torch.empty((rows, self.d), dtype=bf, device=device)
        self.out = torch.empty((tokens, self.d), dtype=bf, device=device)
        self.offsets = torch.empty(self.E + 1, dtype=torch.int64, device=device)
        self.src_index = torch.empty(2 * tokens, dtype=torch.int32, device=device)
        self.experts = torch.empty((tokens, 2), dtype=torch.int32, device=device)
        self.gates = torch.empty((tokens, 2), dtype=torch.float32, device=device)
        self.logits = torch.empty((tokens, self.E), dtype=torch.float32, device=device) if want_logits else None
        self.counts = torch.empty((num_src_shards, self.E), dtype=torch.int32, device=device) if want_counts else None

    def _io(self, x) -> pw_exchange_io:
        io = pw_exchange_io()
        io.src = sharded(x, self.S, self.d, PW_BF16)
        io.dest = None
        io.dst = sharded(self.xd, self.E, self.d, PW_BF16, self.offsets)
        io.src_index = _ptr(self.src_index)
        io.counts = _ptr(self.counts)
        io.b_out = _ptr(self.y)
        io.result = _ptr(self.out)
        io.logits = _ptr(self.logits)
        io.experts = _ptr(self.experts)
        io.gates = _ptr(self.gates)
        return io

    def step(self, x, stream=None) -> pw_future_t:
        """One step with buffers of the static bound (one call)."""
        return self.plan.exchange(self._io(x), stream)

    def split_step(self, x, stream=None) -> pw_future_t:
        """One step in two calls: route (the host waits for the segment
        offsets), allocate the dispatched rows and expert outputs at exactly
        the routed size, then run the rest."""
        import torch
        io = self._io(x)
        offs = self.plan.exchange_begin(io, self.E, stream)
        rows = int(offs[-1])
        self.xd = torch.empty((rows, self.d), dtype=torch.bfloat16, device=self.device)
        self.y = torch.empty((rows, self.d), dtype=torch.bfloat16, device=self.device)
        io.dst = sharded(self.xd, self.E, self.d, PW_BF16, self.offsets)
        io.dst.num_tuples = rows
        io.b_out = _ptr(self.y)
        return self.plan.exchange_end(io, stream)


def _address(t):
    """A tensor's address; an empty tensor has none, and any that is not NULL
    stands for it (nothing is read or written there)."""
    return None if t is None else t.data_ptr() or 256


def _storage(t):
    """Where the memory that a tensor is a part of begins."""
    return None if t is None else t.untyped_storage().data_ptr()


class _Operator:
    """What the plan-less operators share: the device, checked arguments, and
    the workspace and output buffers, made by the first call that needs them,
    on its stream, and kept (so every call returns the same tensors; a call
    that would make them under HIP graph capture is refused: make one call
    before). Calls of one object share its buffers: order them, and keep the
    object until work queued with it on another stream than the first call's,
    or in a graph, is done."""

    def __init__(self, device):
        dev = torch.device(device)
        self.device = torch.device("cuda", torch.cuda.current_device() if dev.index is None else dev.index)
        self._index = self.device.index
        self._buffers = {}
        self._ws_args = (None, 0)  # address and bytes of the workspace; None: not made yet

    def _buf(self, name, shape, dtype, stream):
        b = self._buffers.get(name)
        if b is None:
            capturing = torch.cuda.is_current_stream_capturing()
            # a block that other work of the current stream still uses is no buffer for `stream`
            with torch.cuda.stream(stream):
                if capturing or torch.cuda.is_current_stream_capturing():
                    raise PwError(PW_ERR_STATE, f"the buffer for {name} is made by the first call: make it before capturing")
                b = self._buffers[name] = torch.empty(shape, dtype=dtype, device=self.device)
        return b

    def _workspace(self, sizer, d):
        need = C.c_size_t(0)
        check(sizer(C.byref(d), C.byref(need)))
        if need.value:
            self._ws_bytes, self._ws_args = need.value, None

    def _arg(self, name, t, shape, dtype, or_dtype=None):
        """The address of a tensor that must be contiguous, on this device, of
        this shape and type; None stays None."""
        if t is None:
            return None
        if (t.shape == shape and (t.dtype is dtype or t.dtype is or_dtype) and t.is_contiguous()
                and t.get_device() == self._index):
            return t.data_ptr() or 256  # (see _address)
        raise PwError(PW_ERR_INVALID, f"{name} must be a contiguous {dtype} tensor of shape {shape} on {self.device}, "
                                      f"got {t.dtype} {tuple(t.shape)} on {t.device}")

    def _run(self, fn, d, io, stream, ws=False):
        """ws: whether fn takes the workspace (None: it does, but this call has no use for one)."""
        if ws and self._ws_args is None:
            b = self._buf("workspace", (self._ws_bytes,), torch.uint8, stream)
            self._ws_args = (b.data_ptr(), self._ws_bytes)
        args = self._ws_args if ws else (None, 0) if ws is None else ()
        s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(self._index)
        if torch.cuda.current_device() == self._index:
            check(fn(C.byref(d), C.byref(io), *args, s))
        else:
            with torch.cuda.device(self._index):
                check(fn(C.byref(d), C.byref(io), *args, s))


class RouterBalance(_Operator):
    """Balance loss of a router with per-expert counts, and the gradient of
    its logits (pw_router_balance, pw_router_grad). logits [tokens][E] fp32 and
    experts [tokens][k] int32 as MoE writes them; valid [tokens] bool or uint8
    leaves padding out (None: every token counts)."""

    def __init__(self, tokens, num_experts, top_k=2, balance_coef=1e-2, z_coef=0.0, device="cuda"):
        super().__init__(device)
        self.T, self.E, self.k = tokens, num_experts, top_k
        self._counts = None  # of the last loss() call
        self.desc = pw_balance_desc(tokens, num_experts, top_k, balance_coef, z_coef)
        self._workspace(lib.pw_router_balance_workspace, self.desc)

    def _io(self, logits, experts, valid):
        io = pw_balance_io()
        io.logits = self._arg("logits", logits, (self.T, self.E), torch.float32)
        io.experts = self._arg("experts", experts, (self.T, self.k), torch.int32)
        io.valid = self._arg("valid", valid, (self.T,), torch.bool, torch.uint8)
        return io

    def loss(self, logits, experts, valid=None, stream=None):
        """(counts [E + 1] int32: tuples per expert, then tokens counted;
        prob_mean [E]; loss [2]: balance, z)."""
        io = self._io(logits, experts, valid)
        counts = self._buf("counts", (self.E + 1,), torch.int32, stream)
        mean = self._buf("prob_mean", (self.E,), torch.float32, stream)
        loss = self._buf("loss", (2,), torch.float32, stream)
        io.counts, io.prob_mean, io.loss = _address(counts), _address(mean), _address(loss)
        self._run(lib.pw_router_balance, self.desc, io, stream, ws=True)
        self._counts = counts
        return counts, mean, loss

    def grad(self, logits, experts=None, counts=None, gates=None, dgates=None, valid=None, grad_loss=None, stream=None):
        """dlogits [tokens][E]: of both losses (grad_loss [2], None: ones; counts
        None: those of the last loss() call) and of the gates, if given."""
        io = self._io(logits, experts, valid)
        if counts is None:
            counts = self._counts
        io.counts = self._arg("counts", counts, (self.E + 1,), torch.int32)
        io.gates = self._arg("gates", gates, (self.T, self.k), torch.float32)
        io.dgates = self._arg("dgates", dgates, (self.T, self.k), torch.float32)
        io.grad_loss = self._arg("grad_loss", grad_loss, (2,), torch.float32)
        out = self._buf("dlogits", (self.T, self.E), torch.float32, stream)
        io.dlogits = _address(out)
        self._run(lib.pw_router_grad, self.desc, io, stream)
        return out


class MoEGrad(_Operator):
    """Gradients of an MoE step's combine (pw_moe_combine_grad), and of its
    dispatch and router (pw_moe_dispatch_grad). rows: dispatched rows at most
    (MoE.static_rows). The gradient of the experts' products, from dy to dxd
    in dispatched order, stands between the two calls and is the caller's."""

    def __init__(self, tokens, d, num_experts, rows=None, device="cuda"):
        super().__init__(device)
        self.T, self.d, self.E = tokens, d, num_experts
        self._slot_of = None  # of the last combine() call
        self.rows = 2 * tokens if rows is None else rows
        self.desc = pw_moe_grad_desc(tokens, self.rows, d, num_experts, 2, PW_BF16)
        self._workspace(lib.pw_moe_dispatch_grad_workspace, self.desc)

    def _rows(self, name, t):
        """The descriptor of a call whose dispatched buffers are like t."""
        if t is None or t.dim() != 2:
            raise PwError(PW_ERR_INVALID, f"{name} must be a tensor of shape [rows][d]")
        n = t.shape[0]
        if n > self.rows:
            raise PwError(PW_ERR_INVALID, f"{n} dispatched rows, at most {self.rows}")
        self.desc.rows = n
        return n

    def combine(self, dout, y, gates, src_index, offsets, valid=None, dy=None, stream=None):
        """(dy like y, dgates [tokens][2] fp32, slot_of [tokens][2] int32) from
        the step's y, gates, src_index and offsets. Rows of dy behind
        offsets[E] are left as they are; dy=None: a kept buffer."""
        n = self._rows("y", y)
        bf = torch.bfloat16
        if dy is None:
            dy = self._buf("dy", (self.rows, self.d), bf, stream)[:n]
        dgates = self._buf("dgates", (self.T, 2), torch.float32, stream)
        slot_of = self._buf("slot_of", (self.T, 2), torch.int32, stream)
        if src_index is not None and src_index.dim() == 1 and src_index.shape[0] > n:
            src_index = src_index[:n]
        io = pw_combine_grad_io()
        io.dout = self._arg("dout", dout, (self.T, self.d), bf)
        io.y = self._arg("y", y, (n, self.d), bf)
        io.gates = self._arg("gates", gates, (self.T, 2), torch.float32)
        io.src_index = self._arg("src_index", src_index, (n,), torch.int32)
        io.offsets = self._arg("offsets", offsets, (self.E + 1,), torch.int64)
        io.valid = self._arg("valid", valid, (self.T,), torch.bool, torch.uint8)
        io.dy = self._arg("dy", dy, (n, self.d), bf)
        io.dgates, io.slot_of = _address(dgates), _address(slot_of)
        self._run(lib.pw_moe_combine_grad, self.desc, io, stream)
        self._slot_of = slot_of
        return dy, dgates, slot_of

    def dispatch(self, dxd, dlogits, w_router, x=None, slot_of=None, valid=None, stream=None):
        """(dx [tokens][d] bf16, dw_router [d][E] fp32); slot_of None: that of
        the last combine() call; x None: dx alone (dw_router None)."""
        n = self._rows("dxd", dxd)
        bf = torch.bfloat16
        if slot_of is None:
            slot_of = self._slot_of
        dx = self._buf("dx", (self.T, self.d), bf, stream)
        dw = self._buf("dw_router", (self.d, self.E), torch.float32, stream) if x is not None else None
        io = pw_dispatch_grad_io()
        io.dxd = self._arg("dxd", dxd, (n, self.d), bf)
        io.dlogits = self._arg("dlogits", dlogits, (self.T, self.E), torch.float32)
        io.w_router = self._arg("w_router", w_router, (self.d, self.E), bf)
        io.x = self._arg("x", x, (self.T, self.d), bf)
        io.slot_of = self._arg("slot_of", slot_of, (self.T, 2), torch.int32)
        io.valid = self._arg("valid", valid, (self.T,), torch.bool, torch.uint8)
        io.dx = _address(dx)
        io.dw_router = _address(dw)
        self._run(lib.pw_moe_dispatch_grad, self.desc, io, stream, ws=True)
        return dx, dw


class BlockNorm(_Operator):
    """Norms around a block with its gate and residual scale (pw_block_norm,
    pw_block_norm_grad): r = x_scale x + y_scale gate * norm(y; w_y) closes a
    block, h = norm(r; w_r) opens the next. Tensors given as None drop their
    part out. Rows, weights and gates are of one dtype; gates is the number of
    gate rows, each for rows / gates consecutive rows (0: no gate)."""

    def __init__(self, rows, d, dtype=PW_BF16, gates=0, x_scale=1.0, y_scale=1.0, eps=1e-6, device="cuda"):
        super().__init__(device)
        self.T, self.d, self.G = rows, d, gates
        self.dtype = torch.float32 if dtype == PW_F32 else torch.bfloat16
        self.desc = pw_norm_desc(rows, d, dtype, gates, x_scale, y_scale, eps)
        self._workspace(lib.pw_block_norm_grad_workspace, self.desc)

    def _io(self, y, w_y, gate, w_r):
        io = pw_norm_io()
        io.y = self._arg("y", y, (self.T, self.d), self.dtype)
        io.w_y = self._arg("w_y", w_y, (self.d,), self.dtype)
        io.gate = self._arg("gate", gate, (self.G, self.d), self.dtype)
        io.w_r = self._arg("w_r", w_r, (self.d,), self.dtype)
        return io

    def forward(self, x, y=None, w_y=None, gate=None, w_r=None, r=None, stream=None):
        """(r, h): r is None where y is (the stream is x itself), h where w_r
        is. r may be given (x itself, to update it in place)."""
        io = self._io(y, w_y, gate, w_r)
        io.x = self._arg("x", x, (self.T, self.d), self.dtype)
        if y is None and r is not None:
            raise PwError(PW_ERR_INVALID, "r is written with y only")
        if y is not None and r is None:
            r = self._buf("r", (self.T, self.d), self.dtype, stream)
        h = self._buf("h", (self.T, self.d), self.dtype, stream) if w_r is not None else None
        io.r = self._arg("r", r, (self.T, self.d), self.dtype)
        io.h = _address(h)
        self._run(lib.pw_block_norm, self.desc, io, stream)
        return r, h

    def grad(self, dr=None, dh=None, r=None, y=None, w_y=None, gate=None, w_r=None, valid=None, dx=None, stream=None):
        """(dx, dy, dw_y [d] fp32, dgate [gates][d] fp32, dw_r [d] fp32), None
        where their part is; r: forward's r (with y None: x_scale x). valid
        [rows] bool or uint8: other rows get zeros and add nothing to the
        weights' gradients. dx may be given (dr itself, to update it in place)."""
        rows, f32 = (self.T, self.d), torch.float32
        io = self._io(y, w_y, gate, w_r)
        io.r = self._arg("r", r, rows, self.dtype)
        io.dr = self._arg("dr", dr, rows, self.dtype)
        io.dh = self._arg("dh", dh, rows, self.dtype)
        io.valid = self._arg("valid", valid, (self.T,), torch.bool, torch.uint8)
        if dx is None:
            dx = self._buf("dx", rows, self.dtype, stream)
        io.dx = self._arg("dx", dx, rows, self.dtype)
        dy = self._buf("dy", rows, self.dtype, stream) if y is not None else None
        dw_y = self._buf("dw_y", (self.d,), f32, stream) if w_y is not None else None
        dgate = self._buf("dgate", (self.G, self.d), f32, stream) if gate is not None else None
        dw_r = self._buf("dw_r", (self.d,), f32, stream) if w_r is not None else None
        io.dy, io.dw_y, io.dgate, io.dw_r = _address(dy), _address(dw_y), _address(dgate), _address(dw_r)
        self._run(lib.pw_block_norm_grad, self.desc, io, stream, ws=True)
        return dx, dy, dw_y, dgate, dw_r


class Router(_Operator):
    """Routing of tokens to experts (pw_route) and the gradient of its weights
    (pw_route_grad): softmax or sigmoid scores, a bias that balances the choice,
    groups, top-k, renormalised weights. Padding (valid 0) and places without an
    expert get the id num_experts and the weight 0."""

    def __init__(self, tokens, num_experts, top_k, score="softmax", groups=1, top_groups=1, group_best=2, renorm=True,
                 scale=1.0, device="cuda"):
        super().__init__(device)
        kinds = {"softmax": PW_SCORE_SOFTMAX, "sigmoid": PW_SCORE_SIGMOID}
        if score not in kinds:
            raise PwError(PW_ERR_INVALID, f"score must be one of {sorted(kinds)}, got {score!r}")
        self.T, self.E, self.k = tokens, num_experts, top_k
        self.desc = pw_route_desc(tokens, num_experts, top_k, kinds[score], groups, top_groups, group_best, bool(renorm), scale)

    def _io(self, logits, valid):
        io = pw_route_io()
        io.logits = self._arg("logits", logits, (self.T, self.E), torch.float32)
        io.valid = self._arg("valid", valid, (self.T,), torch.bool, torch.uint8)
        return io

    def forward(self, logits, bias=None, valid=None, stream=None):
        """(experts [tokens][k] int32, best first; weights [tokens][k] fp32)."""
        io = self._io(logits, valid)
        io.bias = self._arg("bias", bias, (self.E,), torch.float32)
        experts = self._buf("experts", (self.T, self.k), torch.int32, stream)
        weights = self._buf("weights", (self.T, self.k), torch.float32, stream)
        io.experts, io.weights = _address(experts), _address(weights)
        self._run(lib.pw_route, self.desc, io, stream)
        return experts, weights

    def grad(self, logits, experts, dweights, valid=None, add=None, stream=None):
        """dlogits [tokens][E] of dweights, with the choice as a constant; add: a
        gradient of the logits that is added (RouterBalance.grad's). dweights[t][j]
        is the caller's: dout[t] . y[t][j] of a combine (MoEGrad.combine gives it
        for two bf16 rows a token, as dgates; there is no operator for more)."""
        io = self._io(logits, valid)
        io.experts = self._arg("experts", experts, (self.T, self.k), torch.int32)
        io.dweights = self._arg("dweights", dweights, (self.T, self.k), torch.float32)
        io.add = self._arg("add", add, (self.T, self.E), torch.float32)
        out = self._buf("dlogits", (self.T, self.E), torch.float32, stream)
        io.dlogits = _address(out)
        self._run(lib.pw_route_grad, self.desc, io, stream)
        return out


def q8_row(d):
    """Bytes of a row of d 8-bit codes (PW_Q8_ROW)."""
    return (d + 63) // 64 * 64


class RowQuant(_Operator):
    """Rows as 8-bit codes with a scale each (pw_quant_rows): tokens, or
    weights [experts * n][d] with a row for each output channel."""

    def __init__(self, rows, d, dtype=PW_BF16, device="cuda"):
        super().__init__(device)
        self.T, self.d = rows, d
        self.dtype = torch.float32 if dtype == PW_F32 else torch.bfloat16
        self.desc = pw_quant_desc(rows, d, dtype)

    def forward(self, x, limit=None, q=None, scale=None, stream=None):
        """(q [rows][q8_row(d)] int8, scale [rows] fp32); q and scale may be given.
        limit: an int64 tensor of one element on the device; rows from there on are
        left as they are."""
        if q is None:
            q = self._buf("q", (self.T, q8_row(self.d)), torch.int8, stream)
        if scale is None:
            scale = self._buf("scale", (self.T,), torch.float32, stream)
        io = pw_quant_io()
        io.x = self._arg("x", x, (self.T, self.d), self.dtype)
        io.limit = self._arg("limit", limit, (1,), torch.int64)
        io.q = self._arg("q", q, (self.T, q8_row(self.d)), torch.int8)
        io.scale = self._arg("scale", scale, (self.T,), torch.float32)
        self._run(lib.pw_quant_rows, self.desc, io, stream)
        return q, scale


class Int8Product(_Operator):
    """Products of dispatched rows with their experts' matrices in 8-bit integers
    (pw_q8_product): out = act(x_scale w_scale (x codes . w codes)). w
    [experts][n][q8_row(d)] int8 with w_scale [experts][n], as RowQuant makes
    them (borrowed: keep them alive). rows: dispatched rows at most. gather k: x
    holds tokens of k tuples each, and src_index[i] // k is the row of dispatched
    row i; scatter: out is in tuple order, row i at src_index[i]."""

    def __init__(self, w, w_scale, d, rows, x_rows=None, gather=0, scatter=False, gelu=False, dtype=PW_BF16, device="cuda"):
        super().__init__(device)
        if w is None or w.dim() != 3:
            raise PwError(PW_ERR_INVALID, "w must be a tensor of shape [experts][n][q8_row(d)]")
        self.E, self.n = w.shape[0], w.shape[1]
        self.d, self.rows = d, rows
        if x_rows is None:
            x_rows = -(-rows // gather) if gather else rows
        self.x_rows = x_rows
        self.dtype = torch.float32 if dtype == PW_F32 else torch.bfloat16
        self.w = (w, w_scale)
        self._w = (self._arg("w", w, (self.E, self.n, q8_row(d)), torch.int8),
                   self._arg("w_scale", w_scale, (self.E, self.n), torch.float32))
        self.desc = pw_q8_desc(rows, x_rows, d, self.n, self.E, dtype, gather, bool(scatter), bool(gelu))
        self._workspace(lib.pw_q8_product_workspace, self.desc)

    def forward(self, x, x_scale=None, offsets=None, src_index=None, out=None, stream=None):
        """out [rows][n]. x [x_rows][d], or its codes [x_rows][q8_row(d)] with
        x_scale [x_rows] (no workspace is made for those). Rows of out that no dispatched row gives are left as they
        are; out=None: a kept buffer."""
        if out is None:
            out = self._buf("out", (self.rows, self.n), self.dtype, stream)
        io = pw_q8_io()
        if x_scale is None:
            io.x = self._arg("x", x, (self.x_rows, self.d), self.dtype)
        else:
            io.q = self._arg("x", x, (self.x_rows, q8_row(self.d)), torch.int8)
            io.q_scale = self._arg("x_scale", x_scale, (self.x_rows,), torch.float32)
        io.w, io.w_scale = self._w
        io.offsets = self._arg("offsets", offsets, (self.E + 1,), torch.int64)
        io.src_index = self._arg("src_index", src_index, (self.rows,), torch.int32)
        io.out = self._arg("out", out, (self.rows, self.n), self.dtype)
        self._run(lib.pw_q8_product, self.desc, io, stream, ws=True if x_scale is None else None)
        return out


class TopkCombine(_Operator):
    """The expert rows of each token, in tuple order, joined by their weights
    (pw_topk_combine): out = add + sum_j weights_j y_j."""

    def __init__(self, tokens, d, top_k, dtype=PW_BF16, device="cuda"):
        super().__init__(device)
        self.T, self.d, self.k = tokens, d, top_k
        self.dtype = torch.float32 if dtype == PW_F32 else torch.bfloat16
        self.desc = pw_combine_desc(tokens, d, top_k, dtype)

    def forward(self, y, weights, add=None, out=None, stream=None):
        """out [tokens][d] from y [tokens * k][d]; a tuple of weight 0 adds nothing.
        out may be given (add itself, to update it in place)."""
        if out is None:
            out = self._buf("out", (self.T, self.d), self.dtype, stream)
        io = pw_topk_combine_io()
        io.y = self._arg("y", y, (self.T * self.k, self.d), self.dtype)
        io.weights = self._arg("weights", weights, (self.T, self.k), torch.float32)
        io.add = self._arg("add", add, (self.T, self.d), self.dtype)
        io.out = self._arg("out", out, (self.T, self.d), self.dtype)
        self._run(lib.pw_topk_combine, self.desc, io, stream)
        return out


class MoEBlock:
    """An MoE step inside a model's block, with its backward pass:

        h = norm(x; w_in);  r = x_scale x + y_scale gate * norm(moe(h); w_out)

    plus the router's balance loss. moe: an MoE with want_logits. w_out and
    gate may be None. The experts' weights are packed when the MoE is built,
    and the gradient of their products is the caller's, between grad_begin
    and grad_end. One forward, then its grad_begin, then grad_end: the buffers
    are the object's, and a call out of this order is refused (grad_begin and
    grad_end may be made again on the same forward)."""

    def __init__(self, moe, w_in, w_out=None, gate=None, x_scale=1.0, y_scale=1.0, eps=1e-6, balance_coef=1e-2,
                 z_coef=0.0):
        if moe.logits is None:
            raise PwError(PW_ERR_INVALID, "the balance loss needs an MoE with want_logits")
        self.moe = moe
        self.w_in, self.w_out, self.gate = w_in, w_out, gate
        device = moe.out.device
        gates = 0 if gate is None else gate.shape[0]
        self.norm_in = BlockNorm(moe.T, moe.d, PW_BF16, eps=eps, device=device)
        self.norm_out = BlockNorm(moe.T, moe.d, PW_BF16, gates, x_scale, y_scale, eps, device)
        self.balance = RouterBalance(moe.T, moe.E, 2, balance_coef, z_coef, device)
        self.grads = MoEGrad(moe.T, moe.d, moe.E, moe.static_rows, device)

        self.h = self._back = None  # of forward; what grad_end takes from grad_begin

    def forward(self, x, valid=None, stream=None):
        """(r, loss [2], counts [E + 1], future of the MoE step); x is kept for the
        backward pass. x may be the r of an earlier call, which is then updated in
        place and leaves no backward pass, but no other buffer that the step writes."""
        m = self.moe
        at = _storage(x)
        if at in [_storage(t) for t in (m.xd, m.y, m.out, self.norm_in._buffers.get("h"))]:
            raise PwError(PW_ERR_INVALID, "x lies in a buffer that the step writes")
        if m.y.shape[0] < m.static_rows:
            raise PwError(PW_ERR_STATE, "the block's step needs an MoE with static buffers")
        self.h = self._back = None  # the step before is over, also if this one fails
        _, h = self.norm_in.forward(x, w_r=self.w_in, stream=stream)
        f = m.step(h, stream)
        counts, _, loss = self.balance.loss(m.logits, m.experts, valid, stream)
        r, _ = self.norm_out.forward(x, y=m.out, w_y=self.w_out, gate=self.gate, stream=stream)
        if at != _storage(r):
            self.x, self.valid, self.h, self._counts = x, valid, h, counts
        return r, loss, counts, f

    def grad_begin(self, dr, stream=None):
        """dy [rows][d], the gradient of the expert outputs moe.y, from dr, that of r."""
        m = self.moe
        if self.h is None:
            raise PwError(PW_ERR_STATE, "grad_begin follows a forward whose x is still there")
        self._back = None
        dx, dout, dw_out, dgate, _ = self.norm_out.grad(dr, y=m.out, w_y=self.w_out, gate=self.gate, valid=self.valid,
                                                        stream=stream)
        dy, dgates, slot_of = self.grads.combine(dout, m.y, m.gates, m.src_index, m.offsets, self.valid, stream=stream)
        self._back = dx, dw_out, dgate, dgates, slot_of
        return dy

    def grad_end(self, dxd, grad_loss=None, stream=None):
        """{"x", "w_in", "w_out", "gate", "w_router"} gradients from dxd, that of the
        dispatched rows moe.xd, and grad_loss [2], that of the losses (None: ones)."""
        m = self.moe
        if self._back is None:
            raise PwError(PW_ERR_STATE, "grad_end follows the grad_begin of the last forward")
        dr, dw_out, dgate, dgates, slot_of = self._back
        dl = self.balance.grad(m.logits, m.experts, self._counts, m.gates, dgates, self.valid, grad_loss, stream)
        dh, dw_router = self.grads.dispatch(dxd, dl, m.w[0], self.h, slot_of, self.valid, stream)
        dx, _, _, _, dw_in = self.norm_in.grad(dr, dh, self.x, w_r=self.w_in, valid=self.valid, stream=stream)
        if _storage(dx) == _storage(self.x):  # x was an earlier call's "x" gradient, whose buffer this one is
            self.h = self._back = None
        return {"x": dx, "w_in": dw_in, "w_out": dw_out, "gate": dgate, "w_router": dw_router}


class Sched:
    """Multi-tenant scheduler: clients with weights submit programs (chain
    runs, exchange steps) that run one after another on the scheduler's own
    stream in proportional shares. Tensors handed to a program are kept
    referenced here until its ticket is waited."""

    def __init__(self, max_inflight=2):
        h = C.c_void_p()
        check(lib.pw_sched_create(max_inflight, C.byref(h)))
        self.handle = h
        self._keep = {}

    def add_client(self, weight=1) -> int:
        c = C.c_uint32(0)
        check(lib.pw_sched_add_client(self.handle, weight, C.byref(c)))
        return c.value

    def _submit(self, client, prog, keep) -> int:
        t = C.c_uint64(0)
        check(lib.pw_sched_submit(self.handle, client, C.byref(prog), C.byref(t)))
        self._keep[t.value] = keep
        return t.value

    def submit_chain(self, client, chain, state, steps, cost=None, aux=None) -> int:
        """A chain run of `steps` steps of `chain` (a Chain) over `state`;
        cost defaults to the step count."""
        prog = pw_program()
        prog.kind = PW_PROG_CHAIN
        prog.cost = steps if cost is None else cost
        prog.plan = chain.plan.handle.value
        prog.steps = steps
        prog.state = sharded(state, chain.N, chain.E, PW_F32)
        prog.aux = _ptr(aux)
        return self._submit(client, prog, (chain, state, aux))

    def submit_exchange(self, client, ex, x, dest, cost=1) -> int:
        """One step of `ex` (an Exchange) on x, dest."""
        prog = pw_program()
        prog.kind = PW_PROG_EXCHANGE
        prog.cost = cost
        prog.plan = ex.plan.handle.value
        prog.io = ex.io(x, dest)
        return self._submit(client, prog, (ex, x, dest))

    def wait(self, ticket, timeout_ns=-1) -> None:
        rc = lib.pw_sched_wait(self.handle, ticket, timeout_ns)
        if rc != PW_ERR_TIMEOUT:  # the ticket is consumed; on a timeout it stays waitable
            self._keep.pop(ticket, None)
        check(rc)

    def hold(self, on=True) -> None:
        check(lib.pw_sched_hold(self.handle, 1 if on else 0))

    def records(self, capacity=1 << 16) -> list:
        """Records of finished programs in dispatch order (each read once):
        (ticket, client, status, dispatch, start_ms, end_ms) tuples."""
        out = []
        buf = (pw_sched_record * capacity)()
        while True:
            n = C.c_size_t(0)
            check(lib.pw_sched_records(self.handle, buf, capacity, C.byref(n)))
            out += [(r.ticket, r.client, r.status, r.dispatch, r.start_ms, r.end_ms) for r in buf[:n.value]]
            if n.value < capacity:
                return out

    def destroy(self) -> None:
        if self.handle:
            check(lib.pw_sched_destroy(self.handle))
            self.handle = None
            self._keep.clear()

    def __del__(self):
        try:
            if getattr(self, "handle", None):
                lib.pw_sched_destroy(self.handle)
        except Exception:
            pass


class _DeviceArray:
    """A borrowed view of device memory for torch.as_tensor (array interface
    of version 2); the memory stays the store's."""

    def __init__(self, ptr, shape, typestr):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr, "data": (ptr, False),
                                         "version": 2, "strides": None}


class Store:
    """HBM object store: owner-labelled device buffers with backpressure."""

    _TYPESTR = {"float32": "<f4", "int32": "<i4", "int64": "<i8", "uint8": "|u1"}

    def __init__(self, nbytes):
        h = C.c_void_p()
        check(lib.pw_store_create(nbytes, C.byref(h)))
        self.handle = h

    def alloc(self, nbytes, owner=0, timeout_ns=-1):
        """(object handle, device address)."""
        obj, ptr = C.c_uint64(0), C.c_void_p()
        check(lib.pw_store_alloc(self.handle, nbytes, owner, timeout_ns, C.byref(obj), C.byref(ptr)))
        return obj.value, ptr.value

    def tensor(self, ptr, shape, dtype="float32"):
        """A torch tensor over store memory (borrowed: valid until freed)."""
        import torch
        return torch.as_tensor(_DeviceArray(ptr, shape, self._TYPESTR[dtype]), device="cuda")

    def free(self, obj, stream=None):
        check(lib.pw_store_free(self.handle, obj, _stream(stream)))

    def release_owner(self, owner, stream=None) -> int:
        n = C.c_uint64(0)
        check(lib.pw_store_release_owner(self.handle, owner, _stream(stream), C.byref(n)))
        return n.value

    def stats(self) -> dict:
        st = pw_store_stats()
        check(lib.pw_store_get_stats(self.handle, C.byref(st)))
        return {name: getattr(st, name) for name, _ in st._fields_}

    def destroy(self):
        if self.handle:
            check(lib.pw_store_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            if getattr(self, "handle", None):
                lib.pw_store_destroy(self.handle)
        except Exception:
            pass
