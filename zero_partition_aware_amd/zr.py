"""ctypes binding of libzr.so (the C ABI in include/zr.h).

Argument marshalling only: every function here turns Python/torch arguments
into the plain pointers and sizes of the C call of the same name, calls it,
and raises ``ZrError`` with the library's message when the status is not
ZR_OK.  No step of the computation happens in Python, and there is no
fallback: if the library is missing the import fails.
"""

import ctypes
import operator
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzr.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built: run `python -m zero_partition_aware_amd.build`")

# torch ships its own HIP runtime under the same soname as ROCm's.  Import it
# first so that the library binds to the runtime torch already holds: two HIP
# runtimes in one process do not share devices, streams or memory.
try:
    import torch  # noqa: F401
except ImportError:
    torch = None
_lib = ctypes.CDLL(LIB_PATH)


def _hip_runtimes_loaded():
    try:
        with open("/proc/self/maps") as fh:
            return sorted({ln.split()[-1] for ln in fh
                           if "libamdhip64" in ln and "/" in ln})
    except OSError:
        return []


if len(_hip_runtimes_loaded()) > 1:
    raise ImportError("two HIP runtimes are loaded in this process "
                      f"({_hip_runtimes_loaded()}); import torch before any "
                      "other HIP library")

ZR_OK, ZR_ERR_INVALID, ZR_ERR_OOM, ZR_ERR_HIP, ZR_ERR_UNSUPPORTED = range(5)
ZR_FP32, ZR_BF16 = 0, 1
ZR_I32, ZR_I64 = 0, 1
ZR_MAX_WORLD = 64
STATUS_NAMES = {0: "ZR_OK", 1: "ZR_ERR_INVALID", 2: "ZR_ERR_OOM",
                3: "ZR_ERR_HIP", 4: "ZR_ERR_UNSUPPORTED"}

c_i64, c_i32, c_vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
c_f64 = ctypes.c_double


class zr_param(ctypes.Structure):
    _fields_ = [("numel", c_i64), ("group", c_i32)]


class zr_group(ctypes.Structure):
    _fields_ = [("world", c_i32), ("sp", c_i32)]


class zr_slice(ctypes.Structure):
    _fields_ = [("bucket", c_i64), ("group", c_i32), ("dst", c_i32),
                ("bucket_offset", c_i64), ("flat_offset", c_i64),
                ("part_offset", c_i64), ("numel", c_i64)]

    def astuple(self):
        return (self.bucket, self.group, self.dst, self.bucket_offset,
                self.flat_offset, self.part_offset, self.numel)


class zr_replica(ctypes.Structure):
    _fields_ = [("ptr", c_vp), ("flat_base", c_i64), ("len", c_i64)]


class zr_adam(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double),
                ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("step", c_i64)]


class zr_linear_grad(ctypes.Structure):
    _fields_ = [("param", c_i64), ("n_out", c_i64), ("n_in", c_i64), ("tokens", c_i64),
                ("dy", c_vp), ("dy_stride", c_i64), ("codes", c_vp), ("scales", c_vp),
                ("in_major", c_i32)]


_P = ctypes.POINTER
_embedding_grad = [c_vp, c_i64, c_i64, c_vp, c_i32, c_i64, ctypes.c_float, c_vp, c_i32, c_i64,
                   c_vp, c_i64, c_i64, c_vp, c_i64, c_vp]
_linear_grads = [c_vp, _P(zr_linear_grad), c_i64, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp]
_products = [c_vp, _P(c_i64), _P(c_i64), c_i64, c_i64, c_i64, c_i32, _P(c_vp), c_vp, c_i64, c_i64,
             c_vp, c_i32, c_i64, c_vp, c_i64, c_vp]
_sigs = {
    "zr_plan_buckets": (c_i32, [_P(zr_param), c_i64, _P(zr_group), c_i32, c_i64,
                                c_i32, c_i64, _P(c_vp)]),
    "zr_plan_free": (None, [c_vp]),
    "zr_plan_num_buckets": (c_i32, [c_vp, _P(c_i64)]),
    "zr_plan_num_params": (c_i32, [c_vp, _P(c_i64)]),
    "zr_plan_partition_gradients": (c_i32, [c_vp, _P(c_i32)]),
    "zr_plan_group_info": (c_i32, [c_vp, c_i32, _P(c_i64), _P(c_i64),
                                   _P(c_i64), _P(ctypes.c_float)]),
    "zr_plan_param_offset": (c_i32, [c_vp, c_i64, _P(c_i64)]),
    "zr_plan_param_partitions": (c_i32, [c_vp, c_i64, _P(_P(c_i32)), _P(c_i32)]),
    "zr_plan_grad_start_offset": (c_i32, [c_vp, c_i64, c_i32, _P(c_i64)]),
    "zr_plan_slices": (c_i32, [c_vp, c_i64, _P(_P(zr_slice)), _P(c_i64)]),
    "zr_plan_param_buckets": (c_i32, [c_vp, c_i64, _P(c_i64), _P(c_i64)]),
    "zr_plan_reduce_launches": (c_i32, [c_vp, c_i32, c_i64, c_i64, c_i32, c_i32, c_i32,
                                        c_i32, _P(c_i64), _P(c_i64)]),
    "zr_reduce_launch_occupancy": (c_i32, [c_i32, c_i32, c_i32, _P(c_i32), _P(c_i32)]),
    "zr_ipg_accumulate": (c_i32, [c_vp, _P(c_i64), _P(c_vp), c_i64, c_i32, c_vp,
                                  c_i64, c_i64, c_vp]),
    "zr_ipg_accumulate_first": (c_i32, [c_vp, _P(c_i64), _P(c_vp), c_i64, c_i32, c_vp,
                                        c_i64, c_i64, c_vp]),
    "zr_reduce_scatter_local": (c_i32, [c_vp, c_i32, c_i64, c_i32, _P(zr_replica),
                                        c_i32, _P(c_vp), c_vp]),
    "zr_reduce_scatter_local_range": (c_i32, [c_vp, c_i32, c_i64, c_i64, c_i32,
                                              _P(zr_replica), c_i32, _P(c_vp), c_vp]),
    "zr_reduce_scatter_adam_range": (c_i32, [c_vp, c_i32, c_i64, c_i64, c_i32,
                                             _P(zr_replica), c_i32, _P(zr_adam), c_vp, c_vp,
                                             c_vp, c_vp, c_vp, c_vp]),
    "zr_copy_grads_in_partition": (c_i32, [c_vp, c_i32, c_i64, c_i32, c_vp, c_vp,
                                           c_vp]),
    "zr_adam_partition": (c_i32, [_P(zr_adam), c_vp, c_vp, c_vp, c_vp, c_vp,
                                  c_i64, c_vp]),
    "zr_reduce_scatter_adam": (c_i32, [c_vp, c_i32, c_i64, c_i32, _P(zr_replica),
                                       c_i32, _P(zr_adam), c_vp, c_vp, c_vp, c_vp,
                                       c_vp, c_vp]),
    "zr_reduce_scatter_adam_capped": (c_i32, [c_vp, c_i32, c_i64, c_i32, _P(zr_replica),
                                              c_i32, _P(zr_adam), c_vp, c_vp, c_vp, c_vp,
                                              c_vp, c_i32, c_vp]),
    "zr_reduce_scatter_adam_noalloc": (c_i32, [c_vp, c_i32, c_i64, c_i32, _P(zr_replica),
                                               c_i32, _P(zr_adam), c_vp, c_vp, c_vp, c_vp,
                                               c_vp, c_vp]),
    "zr_ring_rs_step": (c_i32, [_P(c_vp), c_i32, c_i64, c_i32, c_vp]),
    "zr_ring_ag_step": (c_i32, [_P(c_vp), c_i32, c_i64, c_i32, c_vp]),
    "zr_all_gather_params": (c_i32, [c_vp, c_i32, _P(c_vp), c_i32, c_vp, c_i64, c_i64,
                                     c_vp]),
    "zr_embedding_lookup": (c_i32, [c_vp, c_i64, c_i64, _P(c_vp), c_i32, c_vp, c_i32, c_i64,
                                    ctypes.c_float, c_vp, c_i64, c_vp]),
    "zr_ipg_embedding_workspace": (c_i32, [c_vp, c_i64, c_i64, c_i64, c_i64, c_i64, _P(c_i64)]),
    "zr_ipg_accumulate_embedding": (c_i32, _embedding_grad),
    "zr_ipg_accumulate_embedding_first": (c_i32, _embedding_grad),
    "zr_act_layout": (c_i32, [c_i64, _P(c_i64), _P(c_i64)]),
    "zr_act_quantize": (c_i32, [c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp]),
    "zr_act_dequantize": (c_i32, [c_vp, c_vp, c_i64, c_i64, c_vp, c_i32, c_i64, c_vp]),
    "zr_ipg_linear_workspace": (c_i32, [c_vp, _P(zr_linear_grad), c_i64, c_i64, c_i64,
                                        _P(c_i64)]),
    "zr_ipg_accumulate_linear": (c_i32, _linear_grads),
    "zr_ipg_accumulate_linear_first": (c_i32, _linear_grads),
    "zr_linear_forward_workspace": (c_i32, _products[:7] + [_P(c_i64)]),
    "zr_linear_input_grad_workspace": (c_i32, _products[:7] + [_P(c_i64)]),
    "zr_linear_forward": (c_i32, _products),
    "zr_linear_input_grad": (c_i32, _products),
    "zr_loss_workspace": (c_i32, [c_i64, c_i64, c_i64, c_i32, _P(c_i64)]),
    "zr_distill_loss": (c_i32, [c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i32, c_i64, c_vp, c_i32,
                                c_i64, c_i64, c_vp, c_f64, c_vp, c_vp, c_i64, c_vp, c_i64, c_vp]),
    "zr_policy_loss": (c_i32, [c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp,
                               c_f64, c_f64, c_f64, c_f64, c_vp, c_vp, c_vp, c_i64, c_vp, c_i64, c_vp]),
    "zr_last_error": (ctypes.c_char_p, []),
    "zr_version": (c_i32, []),
}
for _name, (_res, _args) in _sigs.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_sigs)


class ZrError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def _check(status):
    if status != ZR_OK:
        raise ZrError(status, _lib.zr_last_error().decode(errors="replace"))


def zr_last_error():
    return _lib.zr_last_error().decode(errors="replace")


def zr_version():
    return _lib.zr_version()


# ------------------------------------------------------------ marshalling

def _int(x, bits, name):
    """A Python integer for a C int32_t / int64_t argument.  ctypes wraps
    out-of-range values silently (2**32 + 5 would arrive as 5), so the range
    is checked here and a violation raises ZrError(ZR_ERR_INVALID)."""
    if isinstance(x, float) and x.is_integer():
        v = int(x)                      # e.g. reduce_bucket_size=5e8
    else:
        try:
            v = operator.index(x)
        except TypeError:
            raise ZrError(ZR_ERR_INVALID, f"{name} must be an integer, not {x!r}") from None
    lim = 1 << (bits - 1)
    if not -lim <= v < lim:
        raise ZrError(ZR_ERR_INVALID, f"{name} = {v} does not fit in int{bits}_t")
    return v


def _i32(x, name):
    return _int(x, 32, name)


def _i64(x, name):
    return _int(x, 64, name)


def _ptr(t):
    """Device (or host) address of a tensor, or None for None."""
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


_DT_NAME = {ZR_FP32: "fp32", ZR_BF16: "bf16"}


def _buf(t, name, dtype=None, min_numel=None):
    """Checks one buffer argument and returns its address (None for None).

    The C calls see only addresses, so what a pointer cannot carry is checked
    here: a torch tensor must be a contiguous device tensor (a strided view
    would be read as if it were dense), of the element type the call needs,
    and hold at least the elements the call touches.  Violations raise
    ZrError(ZR_ERR_INVALID) before anything is enqueued."""
    if t is None:
        return None
    if torch is not None and isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ZrError(ZR_ERR_INVALID, f"{name} must be contiguous")
        if not t.is_cuda:
            raise ZrError(ZR_ERR_INVALID, f"{name} must be a device tensor")
    if dtype is not None and _dtype_code(t) != dtype:
        raise ZrError(ZR_ERR_INVALID, f"{name} must be {_DT_NAME[dtype]}")
    if min_numel is not None and t.numel() < min_numel:
        raise ZrError(ZR_ERR_INVALID,
                      f"{name} holds {t.numel()} elements; the call touches {min_numel}")
    return ctypes.c_void_p(t.data_ptr())


def _part_numel(plan, group):
    """P_g of the plan's group, queried once per plan and group."""
    P = plan.part_numel.get(group)
    if P is None:
        P = plan.part_numel[group] = zr_plan_group_info(plan, group)[2]
    return P


def _padded_numel(plan, group):
    """L_g = R_g * P_g of the plan's group, queried once per plan and group."""
    key = ("padded", group)
    L = plan.part_numel.get(key)
    if L is None:
        L = plan.part_numel[key] = zr_plan_group_info(plan, group)[1]
    return L


def _world(plan, group):
    """R_g of the plan's group, as given to zr_plan_buckets (an out-of-range
    group is the C call's error: the group query raises it)."""
    g = _i32(group, "group")
    if not 0 <= g < len(plan.worlds):
        zr_plan_group_info(plan, g)
    return plan.worlds[g]


def _expect_len(seq, n, name):
    """The C calls index host arrays by rank: a list shorter (or longer) than
    the group needs would make them read past the array, so its length is
    checked here."""
    if len(seq) != n:
        raise ZrError(ZR_ERR_INVALID, f"{name} has {len(seq)} entries; the call needs {n}")


def _dtype_code(t):
    dt = t.dtype
    if dt is torch.bfloat16:
        return ZR_BF16
    if dt is torch.float32:
        return ZR_FP32
    return -1


def _dtype_name_code(dt):
    """ZR_BF16 / ZR_FP32 for "bf16" / "fp32" or the torch dtype."""
    if dt == "bf16" or (torch is not None and dt is torch.bfloat16):
        return ZR_BF16
    if dt == "fp32" or (torch is not None and dt is torch.float32):
        return ZR_FP32
    raise ZrError(ZR_ERR_INVALID, f"unsupported gradient dtype {dt!r}")


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _adam(lr, beta1, beta2, eps, step):
    return zr_adam(float(lr), float(beta1), float(beta2), float(eps), _i64(step, "step"))


class Plan:
    """Owns a zr_plan handle (freed with zr_plan_free)."""

    def __init__(self, handle, numels=(), worlds=(), param_groups=()):
        self._h = handle
        self.part_numel = {}      # group -> P_g (the plan is immutable)
        self.numels = tuple(int(n) for n in numels)   # param sizes, list order
        self.worlds = tuple(int(w) for w in worlds)   # R_g per group
        self.param_groups = tuple(int(g) for g in param_groups)   # per param

    @property
    def handle(self):
        if not self._h:
            raise ValueError("plan already freed")
        return self._h

    def free(self):
        if self._h:
            _lib.zr_plan_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def zr_plan_buckets(numels, param_groups, groups, reduce_bucket_size,
                    partition_gradients=0, align=1):
    """``groups``: list of (world, sp).  Returns a Plan."""
    n = len(numels)
    params = (zr_param * max(n, 1))()
    for i, (ne, g) in enumerate(zip(numels, param_groups)):
        params[i] = zr_param(_i64(ne, f"numels[{i}]"), _i32(g, f"param_groups[{i}]"))
    gs = (zr_group * max(len(groups), 1))()
    for i, (w, sp) in enumerate(groups):
        gs[i] = zr_group(_i32(w, f"groups[{i}].world"), _i32(sp, f"groups[{i}].sp"))
    out = c_vp()
    _check(_lib.zr_plan_buckets(params, n, gs, _i32(len(groups), "len(groups)"),
                                _i64(reduce_bucket_size, "reduce_bucket_size"),
                                _i32(partition_gradients, "partition_gradients"),
                                _i64(align, "align"),
                                ctypes.byref(out)))
    return Plan(out.value, numels, [w for w, _ in groups], param_groups)


def zr_plan_free(plan):
    plan.free()


def zr_plan_num_buckets(plan):
    v = c_i64()
    _check(_lib.zr_plan_num_buckets(plan.handle, ctypes.byref(v)))
    return v.value


def zr_plan_num_params(plan):
    v = c_i64()
    _check(_lib.zr_plan_num_params(plan.handle, ctypes.byref(v)))
    return v.value


def zr_plan_partition_gradients(plan):
    v = c_i32()
    _check(_lib.zr_plan_partition_gradients(plan.handle, ctypes.byref(v)))
    return v.value


def zr_plan_group_info(plan, g):
    """(total, padded, part_numel, divisor)."""
    t, L, P, d = c_i64(), c_i64(), c_i64(), ctypes.c_float()
    _check(_lib.zr_plan_group_info(plan.handle, _i32(g, "group"), ctypes.byref(t),
                                   ctypes.byref(L), ctypes.byref(P),
                                   ctypes.byref(d)))
    return t.value, L.value, P.value, d.value


def zr_plan_param_offset(plan, p):
    v = c_i64()
    _check(_lib.zr_plan_param_offset(plan.handle, _i64(p, "p"), ctypes.byref(v)))
    return v.value


def zr_plan_param_partitions(plan, p):
    ids, n = _P(c_i32)(), c_i32()
    _check(_lib.zr_plan_param_partitions(plan.handle, _i64(p, "p"), ctypes.byref(ids),
                                         ctypes.byref(n)))
    return [ids[i] for i in range(n.value)]


def zr_plan_grad_start_offset(plan, p, k):
    v = c_i64()
    _check(_lib.zr_plan_grad_start_offset(plan.handle, _i64(p, "p"), _i32(k, "k"),
                                          ctypes.byref(v)))
    return v.value


def zr_plan_param_buckets(plan, p):
    """(first, last) bucket param p feeds."""
    a, b = c_i64(), c_i64()
    _check(_lib.zr_plan_param_buckets(plan.handle, _i64(p, "p"), ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def zr_plan_reduce_launches(plan, group, bucket_first, bucket_count, dst, grad_dtype,
                            fused, with_grad_out=False):
    """(tiles, launches) of a reduce call over buckets [bucket_first,
    bucket_first + bucket_count) for ``dst``; grad_dtype is "bf16" or
    "fp32" (or a torch dtype)."""
    dt = _dtype_name_code(grad_dtype)
    t, n = c_i64(), c_i64()
    _check(_lib.zr_plan_reduce_launches(plan.handle, _i32(group, "group"),
                                        _i64(bucket_first, "bucket_first"),
                                        _i64(bucket_count, "bucket_count"), _i32(dst, "dst"),
                                        dt, int(bool(fused)), int(bool(with_grad_out)),
                                        ctypes.byref(t), ctypes.byref(n)))
    return t.value, n.value


def zr_reduce_launch_occupancy(grad_dtype, fused, world):
    """(workgroups per CU, xcd_weighted) of an uncapped reduce call over
    ``world`` replicas of grad_dtype ("bf16", "fp32" or a torch dtype):
    workgroups per CU 0 = as many as the registers allow; xcd_weighted True
    when the odd XCDs take 31/32 of the even XCDs' tiles."""
    dt = _dtype_name_code(grad_dtype)
    k, w = c_i32(), c_i32()
    _check(_lib.zr_reduce_launch_occupancy(dt, int(bool(fused)), _i32(world, "world"),
                                           ctypes.byref(k), ctypes.byref(w)))
    return k.value, bool(w.value)


def zr_plan_slices(plan, bucket=-1):
    """List of slice tuples (bucket, group, dst, bucket_offset, flat_offset,
    part_offset, numel)."""
    s, n = _P(zr_slice)(), c_i64()
    _check(_lib.zr_plan_slices(plan.handle, _i64(bucket, "bucket"), ctypes.byref(s),
                               ctypes.byref(n)))
    return [s[i].astuple() for i in range(n.value)]


def zr_ipg_accumulate(plan, param_ids, grads, main_grad, window_base=0,
                      window_len=None, stream=None):
    """grads[i]: tensor of param param_ids[i] (bf16 or fp32, all one dtype);
    main_grad: fp32 window tensor."""
    _ipg(_lib.zr_ipg_accumulate, plan, param_ids, grads, main_grad, window_base, window_len,
         stream)


def zr_ipg_accumulate_first(plan, param_ids, grads, main_grad, window_base=0,
                            window_len=None, stream=None):
    """The step's first micro-batch: as zr_ipg_accumulate on a zeroed window,
    without reading (or zeroing) main_grad."""
    _ipg(_lib.zr_ipg_accumulate_first, plan, param_ids, grads, main_grad, window_base,
         window_len, stream)


def _ipg(fn, plan, param_ids, grads, main_grad, window_base, window_len, stream):
    n = len(param_ids)
    if len(grads) != n:
        raise ZrError(ZR_ERR_INVALID, "param_ids and grads differ in length")
    ids = (c_i64 * max(n, 1))(*[_i64(p, f"param_ids[{i}]") for i, p in enumerate(param_ids)])
    dt = _dtype_code(grads[0]) if n else ZR_FP32

    def need(i):
        # the param's size; an out-of-range id is left to the C call's check
        p = ids[i]
        return plan.numels[p] if 0 <= p < len(plan.numels) else None

    ptrs = (c_vp * max(n, 1))(*[_buf(g, f"grads[{i}]", dt, need(i)).value
                                for i, g in enumerate(grads)])
    wl = main_grad.numel() if window_len is None else _i64(window_len, "window_len")
    _check(fn(plan.handle, ids, ptrs, n, dt, _buf(main_grad, "main_grad", ZR_FP32, wl),
              _i64(window_base, "window_base"), wl, _stream(stream)))


def _replicas(reps, plan, group):
    """reps: list of R_g tensors (flat_base 0) or (tensor, flat_base) pairs."""
    _expect_len(reps, _world(plan, group), "reps")
    arr = (zr_replica * max(len(reps), 1))()
    dt = None
    for i, r in enumerate(reps):
        t, base = (r, 0) if not isinstance(r, tuple) else r
        dt = _dtype_code(t) if dt is None else dt
        arr[i] = zr_replica(_buf(t, f"replica {i}", dt).value, _i64(base, f"replica {i} flat_base"),
                            t.numel())
    return arr, (ZR_FP32 if dt is None else dt)


def zr_reduce_scatter_local(plan, group, bucket, dst, reps, part_out,
                            stream=None):
    """part_out: list of fp32 tensors (all destinations when dst == -1, else
    the one partition)."""
    arr, dt = _replicas(reps, plan, group)
    P = _part_numel(plan, group)
    R = _world(plan, group)
    if -1 <= _i32(dst, "dst") < R:        # an out-of-range dst is the C call's error
        _expect_len(part_out, R if int(dst) == -1 else 1, "part_out")
    outs = (c_vp * max(len(part_out), 1))(
        *[_buf(t, f"part_out[{i}]", ZR_FP32, P).value if t is not None else None
          for i, t in enumerate(part_out)])
    _check(_lib.zr_reduce_scatter_local(plan.handle, _i32(group, "group"),
                                        _i64(bucket, "bucket"), _i32(dst, "dst"), arr, dt, outs,
                                        _stream(stream)))


def zr_reduce_scatter_local_range(plan, group, bucket_first, bucket_count, dst, reps,
                                  part_out, stream=None):
    """zr_reduce_scatter_local over buckets [bucket_first, bucket_first +
    bucket_count) in one call."""
    arr, dt = _replicas(reps, plan, group)
    P = _part_numel(plan, group)
    R = _world(plan, group)
    if -1 <= _i32(dst, "dst") < R:        # an out-of-range dst is the C call's error
        _expect_len(part_out, R if int(dst) == -1 else 1, "part_out")
    outs = (c_vp * max(len(part_out), 1))(
        *[_buf(t, f"part_out[{i}]", ZR_FP32, P).value if t is not None else None
          for i, t in enumerate(part_out)])
    _check(_lib.zr_reduce_scatter_local_range(plan.handle, _i32(group, "group"),
                                              _i64(bucket_first, "bucket_first"),
                                              _i64(bucket_count, "bucket_count"),
                                              _i32(dst, "dst"), arr, dt, outs, _stream(stream)))


def zr_reduce_scatter_adam_range(plan, group, bucket_first, bucket_count, dst, reps,
                                 master, m, v, param_bf16=None, grad_out=None, lr=1e-3,
                                 beta1=0.9, beta2=0.999, eps=1e-8, step=1, stream=None):
    """zr_reduce_scatter_adam over buckets [bucket_first, bucket_first +
    bucket_count) in one call."""
    arr, dt = _replicas(reps, plan, group)
    h = _adam(lr, beta1, beta2, eps, step)
    P = _part_numel(plan, group) if int(dst) >= 0 else _padded_numel(plan, group)
    _check(_lib.zr_reduce_scatter_adam_range(plan.handle, _i32(group, "group"),
                                             _i64(bucket_first, "bucket_first"),
                                             _i64(bucket_count, "bucket_count"),
                                             _i32(dst, "dst"), arr, dt, ctypes.byref(h),
                                             _buf(master, "master", ZR_FP32, P),
                                             _buf(m, "m", ZR_FP32, P), _buf(v, "v", ZR_FP32, P),
                                             _buf(param_bf16, "param_bf16", ZR_BF16, P),
                                             _buf(grad_out, "grad_out", ZR_FP32, P),
                                             _stream(stream)))


def zr_copy_grads_in_partition(plan, group, bucket, dst, bucket_layout_src,
                               part_out, stream=None):
    need = 0
    if int(bucket) >= 0:
        for s in zr_plan_slices(plan, bucket):
            if s[1] == int(group) and s[2] == int(dst):
                need = max(need, s[3] + s[6])
    _check(_lib.zr_copy_grads_in_partition(
        plan.handle, _i32(group, "group"), _i64(bucket, "bucket"), _i32(dst, "dst"),
        _buf(bucket_layout_src, "bucket_layout_src", ZR_FP32, need),
        _buf(part_out, "part_out", ZR_FP32, _part_numel(plan, group)), _stream(stream)))


def zr_adam_partition(grad, master, m, v, param_bf16=None, lr=1e-3, beta1=0.9,
                      beta2=0.999, eps=1e-8, step=1, n=None, stream=None):
    h = _adam(lr, beta1, beta2, eps, step)
    nn = master.numel() if n is None else _i64(n, "n")
    need = max(nn, 0)
    _check(_lib.zr_adam_partition(ctypes.byref(h), _buf(grad, "grad", ZR_FP32, need),
                                  _buf(master, "master", ZR_FP32, need),
                                  _buf(m, "m", ZR_FP32, need), _buf(v, "v", ZR_FP32, need),
                                  _buf(param_bf16, "param_bf16", ZR_BF16, need), nn,
                                  _stream(stream)))


def zr_reduce_scatter_adam(plan, group, bucket, dst, reps, master, m, v,
                           param_bf16=None, grad_out=None, lr=1e-3, beta1=0.9,
                           beta2=0.999, eps=1e-8, step=1, stream=None):
    arr, dt = _replicas(reps, plan, group)
    h = _adam(lr, beta1, beta2, eps, step)
    # dst == -1: the state buffers hold every partition (L_g elements)
    P = _part_numel(plan, group) if int(dst) >= 0 else _padded_numel(plan, group)
    _check(_lib.zr_reduce_scatter_adam(plan.handle, _i32(group, "group"),
                                       _i64(bucket, "bucket"), _i32(dst, "dst"), arr, dt,
                                       ctypes.byref(h),
                                       _buf(master, "master", ZR_FP32, P),
                                       _buf(m, "m", ZR_FP32, P), _buf(v, "v", ZR_FP32, P),
                                       _buf(param_bf16, "param_bf16", ZR_BF16, P),
                                       _buf(grad_out, "grad_out", ZR_FP32, P),
                                       _stream(stream)))


def zr_reduce_scatter_adam_capped(plan, group, bucket, dst, reps, master, m, v,
                                  param_bf16=None, grad_out=None, max_workgroups=256,
                                  lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1,
                                  stream=None):
    arr, dt = _replicas(reps, plan, group)
    h = _adam(lr, beta1, beta2, eps, step)
    P = _part_numel(plan, group) if int(dst) >= 0 else _padded_numel(plan, group)
    _check(_lib.zr_reduce_scatter_adam_capped(plan.handle, _i32(group, "group"),
                                              _i64(bucket, "bucket"), _i32(dst, "dst"),
                                              arr, dt, ctypes.byref(h),
                                              _buf(master, "master", ZR_FP32, P),
                                              _buf(m, "m", ZR_FP32, P),
                                              _buf(v, "v", ZR_FP32, P),
                                              _buf(param_bf16, "param_bf16", ZR_BF16, P),
                                              _buf(grad_out, "grad_out", ZR_FP32, P),
                                              _i32(max_workgroups, "max_workgroups"),
                                              _stream(stream)))


def zr_reduce_scatter_adam_noalloc(plan, group, bucket, dst, reps, master, m, v,
                                   param_bf16=None, grad_out=None, lr=1e-3, beta1=0.9,
                                   beta2=0.999, eps=1e-8, step=1, stream=None):
    """zr_reduce_scatter_adam without device allocation: the segment table is
    staged in the library's fixed per-GPU array (calls that overlap on one GPU
    race)."""
    arr, dt = _replicas(reps, plan, group)
    h = _adam(lr, beta1, beta2, eps, step)
    P = _part_numel(plan, group) if int(dst) >= 0 else _padded_numel(plan, group)
    _check(_lib.zr_reduce_scatter_adam_noalloc(plan.handle, _i32(group, "group"),
                                               _i64(bucket, "bucket"), _i32(dst, "dst"), arr,
                                               dt, ctypes.byref(h),
                                               _buf(master, "master", ZR_FP32, P),
                                               _buf(m, "m", ZR_FP32, P),
                                               _buf(v, "v", ZR_FP32, P),
                                               _buf(param_bf16, "param_bf16", ZR_BF16, P),
                                               _buf(grad_out, "grad_out", ZR_FP32, P),
                                               _stream(stream)))


class PreparedReduceScatterAdam:
    """zr_reduce_scatter_adam -- or, with max_workgroups >= 1,
    zr_reduce_scatter_adam_capped -- with its arguments checked and marshalled
    once, for loops that call it per bucket.  Each call passes only the
    bucket, the Adam step and the stream; the C library validates every call
    as usual.  Holds references to the tensors, so their memory stays valid
    while it lives.  One object must not be called from several threads at
    once (the step is written into its argument struct)."""

    def __init__(self, plan, group, dst, reps, master, m, v, param_bf16=None,
                 grad_out=None, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                 max_workgroups=0):
        self._keep = (plan, list(reps), master, m, v, param_bf16, grad_out)
        self._arr, self._dt = _replicas(reps, plan, group)
        self._group = _i32(group, "group")
        self._dst = _i32(dst, "dst")
        P = _part_numel(plan, group) if self._dst >= 0 else _padded_numel(plan, group)
        self._bufs = (_buf(master, "master", ZR_FP32, P), _buf(m, "m", ZR_FP32, P),
                      _buf(v, "v", ZR_FP32, P),
                      _buf(param_bf16, "param_bf16", ZR_BF16, P),
                      _buf(grad_out, "grad_out", ZR_FP32, P))
        self._h = _adam(lr, beta1, beta2, eps, 1)
        self._cap = _i32(max_workgroups, "max_workgroups")
        if self._cap < 0:
            raise ZrError(ZR_ERR_INVALID, "max_workgroups must be >= 0 (0: uncapped)")
        self._handle = plan.handle

    def __call__(self, bucket=-1, step=1, stream=None, count=None):
        """``count`` given: the buckets [bucket, bucket + count) in one call
        (zr_reduce_scatter_adam_range; not with a workgroup cap)."""
        self._h.step = _i64(step, "step")
        b = _i64(bucket, "bucket")
        if count is not None:
            if self._cap:
                raise ZrError(ZR_ERR_INVALID, "a bucket range cannot be capped")
            _check(_lib.zr_reduce_scatter_adam_range(
                self._handle, self._group, b, _i64(count, "count"), self._dst, self._arr,
                self._dt, ctypes.byref(self._h), *self._bufs, _stream(stream)))
            return
        if self._cap:
            _check(_lib.zr_reduce_scatter_adam_capped(
                self._handle, self._group, b, self._dst, self._arr, self._dt,
                ctypes.byref(self._h), *self._bufs, self._cap, _stream(stream)))
        else:
            _check(_lib.zr_reduce_scatter_adam(
                self._handle, self._group, b, self._dst, self._arr, self._dt,
                ctypes.byref(self._h), *self._bufs, _stream(stream)))


def prepare_reduce_scatter_adam(plan, group, dst, reps, master, m, v, param_bf16=None,
                                grad_out=None, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                                max_workgroups=0):
    """A PreparedReduceScatterAdam for these arguments."""
    return PreparedReduceScatterAdam(plan, group, dst, reps, master, m, v, param_bf16,
                                     grad_out, lr, beta1, beta2, eps, max_workgroups)


def zr_ring_rs_step(rank_bufs, chunk_numel, step, stream=None):
    n = len(rank_bufs)
    need = max(int(chunk_numel), 0) * n
    arr = (c_vp * max(n, 1))(*[_buf(t, f"rank_bufs[{i}]", ZR_FP32, need).value
                               if t is not None else None for i, t in enumerate(rank_bufs)])
    _check(_lib.zr_ring_rs_step(arr, n, _i64(chunk_numel, "chunk_numel"), _i32(step, "step"),
                                _stream(stream)))


def zr_ring_ag_step(rank_bufs, chunk_numel, step, stream=None):
    n = len(rank_bufs)
    need = max(int(chunk_numel), 0) * n
    arr = (c_vp * max(n, 1))(*[_buf(t, f"rank_bufs[{i}]", ZR_FP32, need).value
                               if t is not None else None for i, t in enumerate(rank_bufs)])
    _check(_lib.zr_ring_ag_step(arr, n, _i64(chunk_numel, "chunk_numel"), _i32(step, "step"),
                                _stream(stream)))


def zr_all_gather_params(plan, group, parts, out, out_base=0, out_len=None,
                         stream=None):
    """parts: list of R_g partition tensors (bf16 or fp32); out: tensor that
    receives flat elements [out_base, out_base + out_len)."""
    n = len(parts)
    _expect_len(parts, _world(plan, group), "parts")
    dt = _dtype_code(out)
    P = _part_numel(plan, group)
    arr = (c_vp * max(n, 1))(*[(_buf(t, f"parts[{i}]", dt, P).value if t is not None else 0)
                               for i, t in enumerate(parts)])
    ol = out.numel() if out_len is None else _i64(out_len, "out_len")
    _check(_lib.zr_all_gather_params(plan.handle, _i32(group, "group"), arr, dt,
                                     _buf(out, "out", dt, ol), _i64(out_base, "out_base"), ol,
                                     _stream(stream)))


# -------------------------------------------------------- layer operators

# Checks of these calls' tensors.  Each is one condition that holds in every
# good call; what is wrong is only worked out, and named, when it fails.

_FLOATS = None if torch is None else (torch.bfloat16, torch.float32)


def _device_of(t, name):
    """The device of a call's first tensor, which has to be the current one; -2
    (no tensor's) for a host tensor, which the checks that follow refuse."""
    dev = t.get_device()
    if dev < 0:
        return -2
    if dev != torch._C._cuda_getDevice():
        _refuse_device(t, name, torch.cuda.current_device())
    return dev


def _refuse_device(t, name, dev):
    if not t.is_cuda:
        raise ZrError(ZR_ERR_INVALID, f"{name} must be a device tensor")
    raise ZrError(ZR_ERR_INVALID, f"{name} is on device {t.get_device()}, not on the call's "
                                  f"({dev})")


def _rows(t, name, dev, rows=None, cols=None, dtypes=_FLOATS, empty=False):
    """Checks one matrix of contiguous rows (``rows`` x ``cols``, None: any) of
    one of the torch dtypes on the device ``dev`` and returns (address,
    stride).  Rows may lie apart (a slice of wider rows); a strided or
    broadcast column axis is refused (``empty``: unless there are no rows)."""
    shape = t.shape
    if len(shape) == 2 and t.dtype in dtypes and t.get_device() == dev:
        n, c = shape
        stride, step = t.stride()
        if n < 2 and stride < c:
            stride = c
        if ((rows is None or n == rows) and (cols is None or c == cols) and stride >= c and
                (step == 1 or c < 2 or (empty and n == 0))):
            return t.data_ptr(), stride
    if t.dtype not in dtypes:
        raise ZrError(ZR_ERR_INVALID, f"{name} must be one of {dtypes}, not {t.dtype}")
    if len(shape) != 2 or shape[0] != (shape[0] if rows is None else rows) or \
            shape[1] != (shape[1] if cols is None else cols):
        raise ZrError(ZR_ERR_INVALID, f"{name} has shape {tuple(shape)}; the call needs "
                                      f"({'any' if rows is None else rows}, "
                                      f"{'any' if cols is None else cols})")
    if t.get_device() != dev:
        _refuse_device(t, name, dev)
    raise ZrError(ZR_ERR_INVALID, f"{name} must have contiguous rows")


def _dense(t, name, dev, dtype, min_numel=0):
    """Address of a contiguous tensor of the device ``dev``."""
    if (t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and
            t.numel() >= min_numel):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ZrError(ZR_ERR_INVALID, f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        raise ZrError(ZR_ERR_INVALID, f"{name} must be contiguous")
    if t.get_device() != dev:
        _refuse_device(t, name, dev)
    raise ZrError(ZR_ERR_INVALID,
                  f"{name} holds {t.numel()} elements; the call touches {min_numel}")


def _stream_of(stream, dev):
    """The raw handle of ``stream`` or of the device's current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _token_ids(tokens, dev):
    if tokens.dtype is torch.int64:
        return _dense(tokens, "tokens", dev, torch.int64), ZR_I64
    return _dense(tokens, "tokens", dev, torch.int32), ZR_I32


def zr_embedding_lookup(plan, param, dim, parts, tokens, out, scale=1.0, stream=None):
    """out[i] = scale * row tokens[i] of the [vocab, dim] table ``param``,
    read from the R_g partition tensors ``parts`` (bf16 or fp32, those that
    hold none of the table may be None); ids outside [0, vocab) give zeros.
    tokens: int64 or int32, any shape; out: [tokens.numel(), dim]."""
    dev = _device_of(tokens, "tokens")
    ids, wide = _token_ids(tokens, dev)
    n, d, p = tokens.numel(), _i64(dim, "dim"), _i64(param, "param")
    ptr, stride = _rows(out, "out", dev, n, d)
    group = plan.param_groups[p] if 0 <= p < len(plan.param_groups) else 0
    _expect_len(parts, _world(plan, group), "parts")
    P, dtype = _part_numel(plan, group), out.dtype
    arr = (c_vp * len(parts))()
    for k, t in enumerate(parts):
        if t is None:
            continue
        if not (t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and
                t.numel() >= P):
            _dense(t, f"parts[{k}]", dev, dtype, P)
        arr[k] = t.data_ptr()
    status = _lib.zr_embedding_lookup(plan.handle, p, d, arr, dtype is torch.bfloat16, ids, wide,
                                      n, scale, ptr, stride, _stream_of(stream, dev))
    if status:
        _check(status)


def zr_ipg_embedding_workspace(plan, param, dim, n, window_base, window_len):
    """Bytes of workspace the embedding gradient of n tokens needs."""
    v = c_i64()
    _check(_lib.zr_ipg_embedding_workspace(
        plan.handle, _i64(param, "param"), _i64(dim, "dim"), _i64(n, "n"),
        _i64(window_base, "window_base"), _i64(window_len, "window_len"), ctypes.byref(v)))
    return v.value


def zr_ipg_accumulate_embedding(plan, param, dim, tokens, dy, main_grad, workspace,
                                window_base=0, window_len=None, scale=1.0, stream=None):
    """main_grad rows of the table ``param`` += scale * the sums of the rows of
    dy (bf16 or fp32, [tokens.numel(), dim]) over equal ids; ids outside
    [0, vocab) add nothing.  workspace: a uint8 tensor of at least
    zr_ipg_embedding_workspace bytes that no other call uses meanwhile."""
    _embedding(_lib.zr_ipg_accumulate_embedding, plan, param, dim, tokens, dy, main_grad,
               workspace, window_base, window_len, scale, stream)


def zr_ipg_accumulate_embedding_first(plan, param, dim, tokens, dy, main_grad, workspace,
                                      window_base=0, window_len=None, scale=1.0, stream=None):
    """The step's first micro-batch: as zr_ipg_accumulate_embedding on a zeroed
    window, without reading (or zeroing) main_grad."""
    _embedding(_lib.zr_ipg_accumulate_embedding_first, plan, param, dim, tokens, dy, main_grad,
               workspace, window_base, window_len, scale, stream)


def _embedding(fn, plan, param, dim, tokens, dy, main_grad, workspace, window_base, window_len,
               scale, stream):
    dev = _device_of(tokens, "tokens")
    ids, wide = _token_ids(tokens, dev)
    n, d = tokens.numel(), _i64(dim, "dim")
    ptr, stride = _rows(dy, "dy", dev, n, d)
    wl = main_grad.numel() if window_len is None else _i64(window_len, "window_len")
    _check(fn(plan.handle, _i64(param, "param"), d, ids, wide, n, scale, ptr, _dtype_code(dy),
              stride, _dense(main_grad, "main_grad", dev, torch.float32, wl),
              _i64(window_base, "window_base"), wl,
              _dense(workspace, "workspace", dev, torch.uint8), workspace.numel(),
              _stream_of(stream, dev)))


def zr_act_layout(cols):
    """(codes, scales) per row of a checkpoint of ``cols`` columns."""
    c, s = c_i64(), c_i64()
    _check(_lib.zr_act_layout(_i64(cols, "cols"), ctypes.byref(c), ctypes.byref(s)))
    return c.value, s.value


def act_empty(rows, cols, device="cuda"):
    """Uninitialised (codes, scales) for a checkpoint of [rows, cols]: codes
    float8_e4m3fn [rows, cols rounded up to 32], scales uint8 [rows, blocks]."""
    c, s = zr_act_layout(cols)
    return (torch.empty((rows, c), dtype=torch.float8_e4m3fn, device=device),
            torch.empty((rows, s), dtype=torch.uint8, device=device))


_E4M3 = None if torch is None else torch.float8_e4m3fn
_U8 = None if torch is None else torch.uint8


def _checkpoint(codes, scales, dev, rows, cols):
    """Checks a checkpoint's tensors and returns their addresses."""
    blocks = (cols + 31) >> 5
    if (codes.shape == (rows, 32 * blocks) and scales.shape == (rows, blocks) and
            codes.dtype is _E4M3 and scales.dtype is _U8 and codes.get_device() == dev and
            scales.get_device() == dev and codes.is_contiguous() and scales.is_contiguous()):
        return codes.data_ptr(), scales.data_ptr()
    if codes.shape != (rows, 32 * blocks) or scales.shape != (rows, blocks):
        raise ZrError(ZR_ERR_INVALID,
                      f"codes and scales have shapes {tuple(codes.shape)} and "
                      f"{tuple(scales.shape)}; a checkpoint of [{rows}, {cols}] has "
                      f"{(rows, 32 * blocks)} and {(rows, blocks)}")
    return _dense(codes, "codes", dev, _E4M3), _dense(scales, "scales", dev, _U8)


def zr_act_quantize(x, codes, scales, stream=None):
    """The 8-bit checkpoint of x (bf16 or fp32, [rows, cols]) into the tensors
    of act_empty."""
    dev = _device_of(x, "x")
    ptr, stride = _rows(x, "x", dev)
    rows, cols = x.shape
    c, s = _checkpoint(codes, scales, dev, rows, cols)
    status = _lib.zr_act_quantize(ptr, x.dtype is torch.bfloat16, rows, cols, stride, c, s,
                                  _stream_of(stream, dev))
    if status:
        _check(status)


def zr_act_dequantize(codes, scales, out, stream=None):
    """The activations a checkpoint stands for, into out (bf16 or fp32,
    [rows, cols])."""
    dev = _device_of(out, "out")
    ptr, stride = _rows(out, "out", dev)
    rows, cols = out.shape
    c, s = _checkpoint(codes, scales, dev, rows, cols)
    status = _lib.zr_act_dequantize(c, s, rows, cols, ptr, out.dtype is torch.bfloat16, stride,
                                    _stream_of(stream, dev))
    if status:
        _check(status)


def _linear_items(plan, items, dev=None):
    """The items as the C call takes them, on one device (None: the first's)."""
    arr = (zr_linear_grad * max(len(items), 1))()
    for k, (param, dy, codes, scales, *in_major) in enumerate(items):
        if dev is None:
            dev = _device_of(dy, "an item's dy")
        p = _i64(param, "an item's param")
        ptr, stride = _rows(dy, "an item's dy", dev, dtypes=(torch.bfloat16,))
        tokens, n_out = dy.shape
        # an out-of-range id is left to the C call's check
        n_in = plan.numels[p] // max(n_out, 1) if 0 <= p < len(plan.numels) else 1
        c, s = _checkpoint(codes, scales, dev, tokens, max(n_in, 1))
        arr[k] = (p, n_out, n_in, tokens, ptr, stride, c, s,
                  1 if in_major and in_major[0] else 0)
    return arr


def zr_ipg_linear_workspace(plan, items, window_base, window_len):
    """Bytes of workspace zr_ipg_accumulate_linear needs for these items."""
    v = c_i64()
    _check(_lib.zr_ipg_linear_workspace(plan.handle, _linear_items(plan, items),
                                        len(items),
                                        _i64(window_base, "window_base"),
                                        _i64(window_len, "window_len"), ctypes.byref(v)))
    return v.value


def zr_ipg_accumulate_linear(plan, items, main_grad, workspace, window_base=0, window_len=None,
                             stream=None):
    """main_grad of each item's weight += dY^T X^, X^ the activations of an
    8-bit checkpoint.  items: (param, dy, codes, scales) or (..., in_major);
    dy bf16 [tokens, n_out]; in_major True for a weight stored [n_in, n_out].
    workspace: a uint8 tensor of at least zr_ipg_linear_workspace bytes that
    no other call uses meanwhile (None where that is 0)."""
    _linear(_lib.zr_ipg_accumulate_linear, plan, items, main_grad, workspace, window_base,
            window_len, stream)


def zr_ipg_accumulate_linear_first(plan, items, main_grad, workspace, window_base=0,
                                   window_len=None, stream=None):
    """The step's first micro-batch: as zr_ipg_accumulate_linear on a zeroed
    window, without reading (or zeroing) main_grad."""
    _linear(_lib.zr_ipg_accumulate_linear_first, plan, items, main_grad, workspace, window_base,
            window_len, stream)


def _linear(fn, plan, items, main_grad, workspace, window_base, window_len, stream):
    dev = _device_of(main_grad, "main_grad")
    wl = main_grad.numel() if window_len is None else _i64(window_len, "window_len")
    arr = _linear_items(plan, items, dev)
    ws = None if workspace is None else _dense(workspace, "workspace", dev, torch.uint8)
    _check(fn(plan.handle, arr, len(items),
              _dense(main_grad, "main_grad", dev, torch.float32, wl),
              _i64(window_base, "window_base"), wl, ws,
              0 if workspace is None else workspace.numel(), _stream_of(stream, dev)))


def _scratch(workspace, dev):
    if workspace is None:
        return None, 0
    return _dense(workspace, "workspace", dev, torch.uint8), workspace.numel()


_LIM64 = 1 << 63


def _group_list(plan, params, counts):
    """The params and their counts as the C call takes them."""
    n = len(params)
    _expect_len(counts, n, "counts")
    try:
        lists = (c_i64 * max(n, 1))(*params), (c_i64 * max(n, 1))(*counts), n
    except TypeError:
        raise ZrError(ZR_ERR_INVALID, "params and counts must be integers") from None
    # ctypes keeps the low 64 bits of what does not fit
    if n and (min(params) < -_LIM64 or max(params) >= _LIM64):
        raise ZrError(ZR_ERR_INVALID, "params must fit in int64_t")
    if n and (min(counts) < -_LIM64 or max(counts) >= _LIM64):
        raise ZrError(ZR_ERR_INVALID, "counts must fit in int64_t")
    return lists


def zr_linear_forward_workspace(plan, params, counts, n_out, n_in, in_major=False):
    """Bytes of workspace zr_linear_forward needs for these params and counts."""
    p, c, n = _group_list(plan, params, counts)
    v = c_i64()
    _check(_lib.zr_linear_forward_workspace(plan.handle, p, c, n, _i64(n_out, "n_out"),
                                            _i64(n_in, "n_in"), bool(in_major), ctypes.byref(v)))
    return v.value


def zr_linear_input_grad_workspace(plan, params, counts, n_out, n_in, in_major=False):
    """Bytes of workspace zr_linear_input_grad needs for these params and counts."""
    p, c, n = _group_list(plan, params, counts)
    v = c_i64()
    _check(_lib.zr_linear_input_grad_workspace(plan.handle, p, c, n, _i64(n_out, "n_out"),
                                               _i64(n_in, "n_in"), bool(in_major),
                                               ctypes.byref(v)))
    return v.value


def zr_linear_forward(plan, params, counts, parts, x, y, in_major=False, workspace=None,
                      stream=None):
    """y = x W^T, the first counts[0] rows with the weight params[0], the next
    counts[1] with params[1], and so on (experts, their rows sorted), each
    weight read from the R_g bf16 partition tensors ``parts`` (those that hold
    none of them may be None).  x: bf16 [rows, n_in]; y: bf16 or fp32 [rows,
    n_out]; in_major True for weights stored [n_in, n_out].  Rows behind the
    last count stay as they are.  workspace: a uint8 tensor of at least
    zr_linear_forward_workspace bytes that no other call uses meanwhile (None
    where that is 0)."""
    _product(_lib.zr_linear_forward, plan, params, counts, parts, x, "x", y, "y", False, in_major,
             workspace, stream)


def zr_linear_input_grad(plan, params, counts, parts, dy, dx, in_major=False, workspace=None,
                         stream=None):
    """dx = dy W, grouped as in zr_linear_forward.  dy: bf16 [rows, n_out]; dx:
    bf16 or fp32 [rows, n_in]."""
    _product(_lib.zr_linear_input_grad, plan, params, counts, parts, dy, "dy", dx, "dx", True,
             in_major, workspace, stream)


def _product(fn, plan, params, counts, parts, x, x_name, y, y_name, swap, in_major, workspace,
             stream):
    dev = _device_of(x, x_name)
    xp, xs = _rows(x, x_name, dev, dtypes=(torch.bfloat16,), empty=True)
    rows, depth = x.shape
    yp, ys = _rows(y, y_name, dev, rows, empty=True)
    cols = y.shape[1]
    p, c, n = _group_list(plan, params, counts)
    first = params[0] if n else 0
    # an out-of-range id is left to the C call's check
    group = plan.param_groups[first] if 0 <= first < len(plan.param_groups) else 0
    _expect_len(parts, _world(plan, group), "parts")
    P = _part_numel(plan, group)
    arr = (c_vp * len(parts))()
    for k, t in enumerate(parts):
        if t is None:
            continue
        if not (t.dtype is torch.bfloat16 and t.get_device() == dev and t.is_contiguous() and
                t.numel() >= P):
            _dense(t, f"parts[{k}]", dev, torch.bfloat16, P)
        arr[k] = t.data_ptr()
    ws, nbytes = _scratch(workspace, dev)
    status = fn(plan.handle, p, c, n, depth if swap else cols, cols if swap else depth,
                bool(in_major), arr, xp, rows, xs, yp, y.dtype is torch.bfloat16, ys, ws, nbytes,
                _stream_of(stream, dev))
    if status:
        _check(status)


def zr_loss_workspace(rows, vocab, top, dtype):
    """Bytes of workspace that a loss over [rows, vocab] logits of the torch
    ``dtype`` needs, with ``top`` entries a row (1 for the policy loss)."""
    v = c_i64()
    _check(_lib.zr_loss_workspace(_i64(rows, "rows"), _i64(vocab, "vocab"), _i64(top, "top"),
                                  _dtype_name_code(dtype), ctypes.byref(v)))
    return v.value


def _loss_rows(logits, dlogits, dev):
    """(address, stride) of the logits and of the gradient (null, vocab)."""
    z = _rows(logits, "logits", dev, empty=True)
    rows, vocab = logits.shape
    if dlogits is None:
        return z, (None, vocab)
    return z, _rows(dlogits, "dlogits", dev, rows, vocab, (logits.dtype,), empty=True)


def _per_row(t, name, dev, rows):
    """Address of one fp32 a row (None: null)."""
    if t is None:
        return None
    if t.shape != (rows,):
        raise ZrError(ZR_ERR_INVALID, f"{name} has shape {tuple(t.shape)}; the call needs ({rows},)")
    return _dense(t, name, dev, torch.float32)


_IDS = None if torch is None else (torch.int64, torch.int32)


def zr_distill_loss(logits, ids, teacher, weight, loss, dlogits=None, temperature=1.0,
                    workspace=None, stream=None):
    """Each row's distillation loss from a teacher's top logits, and its
    gradient.  logits: bf16 or fp32 [rows, vocab]; ids (int64 or int32) and
    teacher (bf16 or fp32): [rows, top], the teacher's columns and logits, ids
    outside [0, vocab) for none; weight: fp32 [rows] or None (1); loss: fp32
    [rows]; dlogits: like logits, logits itself, or None.  workspace: a uint8
    tensor of at least zr_loss_workspace bytes that no other call uses meanwhile
    (None where that is 0)."""
    dev = _device_of(logits, "logits")
    (z, zs), (g, gs) = _loss_rows(logits, dlogits, dev)
    rows, vocab = logits.shape
    i, istride = _rows(ids, "ids", dev, rows, None, _IDS, empty=True)
    top = ids.shape[1]
    t, tstride = _rows(teacher, "teacher", dev, rows, top, empty=True)
    ws, nbytes = _scratch(workspace, dev)
    _check(_lib.zr_distill_loss(
        z, logits.dtype is torch.bfloat16, rows, vocab, zs, i, ids.dtype is torch.int64, istride,
        t, teacher.dtype is torch.bfloat16, tstride, top, _per_row(weight, "weight", dev, rows),
        temperature, _per_row(loss, "loss", dev, rows), g, gs, ws, nbytes, _stream_of(stream, dev)))


def zr_policy_loss(logits, tokens, old_logp, ref_logp, advantage, weight, loss, logp,
                   dlogits=None, clip_low=0.2, clip_high=0.2, kl=0.0, temperature=1.0,
                   workspace=None, stream=None):
    """Each row's clipped policy loss with a KL term, its token's
    log-probability, and its gradient.  logits: bf16 or fp32 [rows, vocab];
    tokens: int64 or int32 [rows], outside [0, vocab) for padding; old_logp,
    advantage, and ref_logp (None where kl is 0), weight (None: 1): fp32 [rows];
    loss, logp: fp32 [rows]; dlogits: like logits, logits itself, or None.
    workspace: as in zr_distill_loss, for top 1."""
    dev = _device_of(logits, "logits")
    (z, zs), (g, gs) = _loss_rows(logits, dlogits, dev)
    rows, vocab = logits.shape
    if tokens.shape != (rows,):
        raise ZrError(ZR_ERR_INVALID,
                      f"tokens has shape {tuple(tokens.shape)}; the call needs ({rows},)")
    a, wide = _token_ids(tokens, dev)
    ws, nbytes = _scratch(workspace, dev)
    _check(_lib.zr_policy_loss(
        z, logits.dtype is torch.bfloat16, rows, vocab, zs, a, wide,
        _per_row(old_logp, "old_logp", dev, rows), _per_row(ref_logp, "ref_logp", dev, rows),
        _per_row(advantage, "advantage", dev, rows), _per_row(weight, "weight", dev, rows),
        clip_low, clip_high, kl, temperature, _per_row(loss, "loss", dev, rows),
        _per_row(logp, "logp", dev, rows), g, gs, ws, nbytes, _stream_of(stream, dev)))
