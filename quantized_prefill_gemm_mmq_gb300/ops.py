"""Thin PyTorch binding over libmmq's C ABI (argument marshalling only).

Every function checks device, dtype, shape and contiguity, passes raw device
pointers and the current CUDA stream to the library, and raises MMQError on
a non-zero status.  No arithmetic of the method happens here.
"""
from __future__ import annotations

import ctypes
import math

import torch

from ._lib import KVCacheC, MMQError, load

BLOCK_BYTES = {"q4_K": 144, "q6_K": 210, "q5_K": 176, "q8_0": 272}   # bytes per 256 weights of a row


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(t.data_ptr() if t is not None else 0)


def _check(call: str, status: int):
    if status != 0:
        raise MMQError(call, status)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libmmq ops need CUDA tensors")


def quantize_q8_1(x: torch.Tensor, want_qs: bool = True, want_xh: bool = True, want_xa: bool = True, out=None):
    """q8_1-quantise activations x [T][K] f32 (row stride may exceed K).

    Returns (qs, ds, xh, xa):
      qs  int8 [T][K] values, or None;
      ds  int32 [T][K/32] holding the uint32 words (f16 d | int16 block sum);
      xh  float16 [T][K], the same integer values as f16 (per-sub-block operand), or None;
      xa  float16 [2][T][K], the dequantised values f32(d)*q as exact hi + lo planes
          (production operand), or None.
    `out` may supply the four buffers (any of qs / xh / xa may be None).
    """
    _need_cuda(x)
    if x.dtype != torch.float32 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D float32 tensor with unit column stride")
    T, K = x.shape
    dev = x.device
    if out is not None:
        qs, ds, xh, xa = out
        for t, dt, shape in ((qs, torch.int8, (T, K)), (ds, torch.int32, (T, K // 32)),
                             (xh, torch.float16, (T, K)), (xa, torch.float16, (2, T, K))):
            if t is not None and (t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous()):
                raise ValueError("bad output buffer")
        if ds is None:
            raise ValueError("ds buffer required")
    else:
        qs = torch.empty((T, K), dtype=torch.int8, device=dev) if want_qs else None
        xh = torch.empty((T, K), dtype=torch.float16, device=dev) if want_xh else None
        xa = torch.empty((2, T, K), dtype=torch.float16, device=dev) if want_xa else None
        ds = torch.empty((T, K // 32), dtype=torch.int32, device=dev)
    _need_cuda(qs, ds, xh, xa)
    with torch.cuda.device(dev):
        st = load().mmq_quantize_q8_1(_ptr(x), x.stride(0), T, K, _ptr(qs), _ptr(ds), _ptr(xh), _ptr(xa),
                                      _stream(dev))
    _check("mmq_quantize_q8_1", st)
    return qs, ds, xh, xa


def _check_gemm_args(fmt: str, w: torch.Tensor, xv: torch.Tensor, O: int, planes: int):
    _need_cuda(w, xv)
    if fmt not in BLOCK_BYTES:
        raise ValueError(f"unknown format {fmt!r}")
    if xv.dtype != torch.float16 or xv.dim() != (2 if planes == 1 else 3) or not xv.is_contiguous() or \
            (planes == 2 and xv.shape[0] != 2):
        raise ValueError("activation operand must be contiguous float16 [T][K] (xh) or [2][T][K] (xa)")
    T, K = xv.shape[-2:]
    if w.dtype != torch.uint8 or not w.is_contiguous() or w.numel() != O * (K // 256) * BLOCK_BYTES[fmt]:
        raise ValueError("w must be contiguous uint8 holding O*(K/256) super-blocks")
    if w.device != xv.device:
        raise ValueError("w and the activations must be on the same device")
    return T, K


def _out(out, T, O, dev):
    if out is None:
        return torch.empty((T, O), dtype=torch.float32, device=dev)
    if out.dtype != torch.float32 or tuple(out.shape) != (T, O) or not out.is_contiguous():
        raise ValueError("out must be contiguous float32 [T][O]")
    return out


def _check_ds(ds, T, K):
    if ds.dtype != torch.int32 or tuple(ds.shape) != (T, K // 32) or not ds.is_contiguous():
        raise ValueError("ds must be contiguous int32 [T][K/32]")


def gemm(fmt: str, w: torch.Tensor, xa: torch.Tensor, ds: torch.Tensor, O: int,
         out: torch.Tensor | None = None) -> torch.Tensor:
    """Production GEMM: Y [T][O] f32 from W (`fmt`: q4_K, q5_K or q6_K) and the xa/ds
    activation planes (q6_K does not read ds)."""
    T, K = _check_gemm_args(fmt, w, xa, O, planes=2)
    _check_ds(ds, T, K)
    out = _out(out, T, O, xa.device)
    fn = {"q4_K": load().mmq_gemm_q4K, "q6_K": load().mmq_gemm_q6K, "q5_K": load().mmq_gemm_q5K}.get(fmt)
    if fn is None:
        raise ValueError(f"no production GEMM for {fmt!r} (q8_0: gemm_subblock)")
    with torch.cuda.device(xa.device):
        st = fn(_ptr(w), _ptr(xa), _ptr(ds), _ptr(out), T, O, K, _stream(xa.device))
    _check(f"gemm({fmt})", st)
    return out


SMALL_T_MAX = 64          # mmq_gemm_q4K_small
SMALL_IMMA_T_MAX = 16     # mmq_gemm_q4K_small_imma


def gemm_small(w: torch.Tensor, xa: torch.Tensor, ds: torch.Tensor, O: int,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """q4_K GEMM for T <= 64 tokens (weight rows on the tensor core's 128-row
    side, fed from tensor memory); same operands and result as gemm("q4_K")."""
    T, K = _check_gemm_args("q4_K", w, xa, O, planes=2)
    _check_ds(ds, T, K)
    out = _out(out, T, O, xa.device)
    with torch.cuda.device(xa.device):
        st = load().mmq_gemm_q4K_small(_ptr(w), _ptr(xa), _ptr(ds), _ptr(out), T, O, K, _stream(xa.device))
    _check("mmq_gemm_q4K_small", st)
    return out


def gemm_small_imma(w: torch.Tensor, qs: torch.Tensor, ds: torch.Tensor, O: int,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """q4_K GEMM for T <= 16 tokens on the int8 warp MMA from the int8 q8_1 values qs [T][K] and ds."""
    _need_cuda(w, qs)
    if qs.dtype != torch.int8 or qs.dim() != 2 or not qs.is_contiguous():
        raise ValueError("qs must be contiguous int8 [T][K]")
    T, K = qs.shape
    if w.dtype != torch.uint8 or not w.is_contiguous() or w.numel() != O * (K // 256) * BLOCK_BYTES["q4_K"]:
        raise ValueError("w must be contiguous uint8 holding O*(K/256) q4_K super-blocks")
    _check_ds(ds, T, K)
    out = _out(out, T, O, qs.device)
    with torch.cuda.device(qs.device):
        st = load().mmq_gemm_q4K_small_imma(_ptr(w), _ptr(qs), _ptr(ds), _ptr(out), T, O, K, _stream(qs.device))
    _check("mmq_gemm_q4K_small_imma", st)
    return out


GEMV_T_MAX = 16           # mmq_gemv_q4K, mmq_gemv_q6K


def gemv(w: torch.Tensor, xh: torch.Tensor, ds: torch.Tensor, O: int,
         out: torch.Tensor | None = None, fmt: str = "q4_K") -> torch.Tensor:
    """Decode-shaped product for T <= 16 tokens from the f16 copies of the int8
    q8_1 values xh [T][K] and ds (per-sub-block integer dots on the f16 warp
    MMA), W in q4_K or q6_K; same result as gemm(fmt) up to f32 summation order."""
    T, K = _check_gemm_args(fmt, w, xh, O, planes=1)
    _check_ds(ds, T, K)
    out = _out(out, T, O, xh.device)
    fn = load().mmq_gemv_q4K if fmt == "q4_K" else load().mmq_gemv_q6K
    with torch.cuda.device(xh.device):
        st = fn(_ptr(w), _ptr(xh), _ptr(ds), _ptr(out), T, O, K, _stream(xh.device))
    _check(f"gemv({fmt})", st)
    return out


DECODE_T_MAX = 4          # mmq_gemv_q4K_f32
DECODE_K_MAX = 32768


def gemv_f32(w: torch.Tensor, x: torch.Tensor, O: int, out: torch.Tensor | None = None,
             fmt: str = "q4_K") -> torch.Tensor:
    """Decode-shaped product for T <= 4 f32 tokens x [T][K] with the q8_1
    quantisation built into the kernel (no quantise launch), W in q4_K or q6_K;
    same result as gemm(fmt) on quantize_q8_1(x) up to f32 summation order."""
    _need_cuda(w, x)
    if x.dim() != 2 or x.dtype != torch.float32 or x.stride(1) != 1:
        raise ValueError("x must be a row-major f32 [T][K] tensor")
    T, K = x.shape
    if fmt not in ("q4_K", "q6_K"):
        raise ValueError(f"no decode product for {fmt!r}")
    if w.dtype != torch.uint8 or w.numel() != O * (K // 256) * BLOCK_BYTES[fmt]:
        raise ValueError(f"w must hold O*(K/256) {fmt} super-blocks (uint8)")
    out = _out(out, T, O, x.device)
    fn = load().mmq_gemv_q4K_f32 if fmt == "q4_K" else load().mmq_gemv_q6K_f32
    with torch.cuda.device(x.device):
        st = fn(_ptr(w), _ptr(x), x.stride(0), _ptr(out), T, O, K, _stream(x.device))
    _check(f"gemv_f32({fmt})", st)
    return out


def interleave_gate_up(w_gate: torch.Tensor, w_up: torch.Tensor, F: int) -> torch.Tensor:
    """The weight layout of gemm_swiglu: gate and up q4_K rows interleaved in groups
    of 64 rows (a permutation of whole rows; no arithmetic)."""
    if w_gate.shape != w_up.shape or w_gate.dtype != torch.uint8 or w_gate.numel() % F or F % 64:
        raise ValueError("gate and up must be uint8 buffers of F rows each, F % 64 == 0")
    rb = w_gate.numel() // F
    g = w_gate.reshape(F // 64, 64, rb)
    u = w_up.reshape(F // 64, 64, rb)
    return torch.cat([g, u], dim=1).reshape(-1).contiguous()


def gemm_swiglu(w_gu: torch.Tensor, xa: torch.Tensor, ds: torch.Tensor, F: int, out=None, want_qs: bool = True):
    """h = silu(X W_gate^T) * (X W_up^T) quantised to q8_1, from the interleaved
    gate/up weights (interleave_gate_up) and the input's xa/ds planes.
    Returns (qs or None, ds, xa) of h [T][F]: the operands of the down projection."""
    T, K = _check_gemm_args("q4_K", w_gu, xa, 2 * F, planes=2)
    _check_ds(ds, T, K)
    dev = xa.device
    if out is not None:
        hq, hd, hx = out
        if hd is None or hx is None:
            raise ValueError("ds and xa buffers required")
        for t, dt, shape in ((hq, torch.int8, (T, F)), (hd, torch.int32, (T, F // 32)), (hx, torch.float16, (2, T, F))):
            if t is not None and (t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous()):
                raise ValueError("bad output buffer")
    else:
        hq = torch.empty((T, F), dtype=torch.int8, device=dev) if want_qs else None
        hd = torch.empty((T, F // 32), dtype=torch.int32, device=dev)
        hx = torch.empty((2, T, F), dtype=torch.float16, device=dev)
    with torch.cuda.device(dev):
        st = load().mmq_gemm_q4K_swiglu(_ptr(w_gu), _ptr(xa), _ptr(ds), _ptr(hx), _ptr(hd), _ptr(hq), T, F, K,
                                        _stream(dev))
    _check("mmq_gemm_q4K_swiglu", st)
    return hq, hd, hx


def splitk_sizes(T: int, O: int, K: int, ksplit: int) -> tuple[int, int]:
    """(floats of partial-sum workspace, ints of tile counters) for a split-K q4_K GEMM."""
    pf, nc = ctypes.c_int64(0), ctypes.c_int64(0)
    _check("mmq_splitk_sizes", load().mmq_splitk_sizes(T, O, K, ksplit, ctypes.byref(pf), ctypes.byref(nc)))
    return pf.value, nc.value


_SM_COUNT: dict[int, int] = {}


def sm_count(device: torch.device | int | None = None) -> int:
    """Streaming multiprocessors of a CUDA device (the current one by default)."""
    idx = torch.cuda.current_device() if device is None else torch.device("cuda", device).index \
        if isinstance(device, int) else (device.index if device.index is not None else torch.cuda.current_device())
    if idx not in _SM_COUNT:
        _SM_COUNT[idx] = torch.cuda.get_device_properties(idx).multi_processor_count
    return _SM_COUNT[idx]


def choose_ksplit(T: int, O: int, K: int, sms: int | None = None) -> int:
    """Splits of K that bring the grid near one wave when the output has few
    tiles; `sms` defaults to the current device's SM count."""
    if sms is None:
        sms = sm_count()
    tiles = -(-O // 128) * -(-T // 128)
    return max(1, min(K // 256, sms // max(1, tiles)))


class SplitKWorkspace:
    """Caller-owned scratch of the split-K q4_K GEMM: partial sums and tile
    counters (the counters start at zero and every call leaves them at zero).
    Calls that share one workspace must be ordered (one stream)."""

    def __init__(self, device, max_partial_floats: int, max_tiles: int):
        self.part = torch.empty(max(1, max_partial_floats), dtype=torch.float32, device=device)
        self.counters = torch.zeros(max(1, max_tiles), dtype=torch.int32, device=device)

    def fits(self, partial_floats: int, tiles: int) -> bool:
        return partial_floats <= self.part.numel() and tiles <= self.counters.numel()


def gemm_splitk(w: torch.Tensor, xa: torch.Tensor, ds: torch.Tensor, O: int, ksplit: int | None = None,
                workspace: SplitKWorkspace | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """q4_K production GEMM with K split over `ksplit` CTAs per output tile (default:
    choose_ksplit); partial sums are added in a fixed order, so results repeat bit
    for bit.  Without `workspace` one is allocated for this call."""
    T, K = _check_gemm_args("q4_K", w, xa, O, planes=2)
    _check_ds(ds, T, K)
    out = _out(out, T, O, xa.device)
    if ksplit is None:
        ksplit = choose_ksplit(T, O, K)
    pf, nc = splitk_sizes(T, O, K, ksplit)
    if workspace is None or not workspace.fits(pf, nc):
        workspace = SplitKWorkspace(xa.device, pf, nc)
    with torch.cuda.device(xa.device):
        st = load().mmq_gemm_q4K_splitk(_ptr(w), _ptr(xa), _ptr(ds), _ptr(out), T, O, K, ksplit,
                                        _ptr(workspace.part), _ptr(workspace.counters), _stream(xa.device))
    _check("mmq_gemm_q4K_splitk", st)
    return out


def gemm_splitk_static(w: torch.Tensor, xa: torch.Tensor, ds: torch.Tensor, O: int, ksplit: int | None = None,
                       out: torch.Tensor | None = None) -> torch.Tensor:
    """gemm_splitk with the library's static scratch (no workspace anywhere);
    calls on one device must not overlap in time."""
    T, K = _check_gemm_args("q4_K", w, xa, O, planes=2)
    _check_ds(ds, T, K)
    out = _out(out, T, O, xa.device)
    if ksplit is None:
        ksplit = choose_ksplit(T, O, K)
    with torch.cuda.device(xa.device):
        st = load().mmq_gemm_q4K_splitk_static(_ptr(w), _ptr(xa), _ptr(ds), _ptr(out), T, O, K, ksplit,
                                               _stream(xa.device))
    _check("mmq_gemm_q4K_splitk_static", st)
    return out


def gemm_subblock(fmt: str, w: torch.Tensor, xh: torch.Tensor, ds: torch.Tensor, O: int,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Per-sub-block GEMM (exact integer sub-block dots + f32 fold) from the xh/ds planes;
    `fmt` q4_K, q5_K, q6_K or q8_0 (q8_0's only form)."""
    T, K = _check_gemm_args(fmt, w, xh, O, planes=1)
    _check_ds(ds, T, K)
    out = _out(out, T, O, xh.device)
    fn = {"q4_K": load().mmq_gemm_q4K_subblock, "q6_K": load().mmq_gemm_q6K_subblock,
          "q5_K": load().mmq_gemm_q5K_subblock, "q8_0": load().mmq_gemm_q8_0}[fmt]
    with torch.cuda.device(xh.device):
        st = fn(_ptr(w), _ptr(xh), _ptr(ds), _ptr(out), T, O, K, _stream(xh.device))
    _check(f"gemm_subblock({fmt})", st)
    return out


def debug_subdots(fmt: str, w: torch.Tensor, xh: torch.Tensor, O: int) -> torch.Tensor:
    """Per-sub-block integer dots: int32 [T][O][K/16] (q6_K) or [T][O][K/32] (the others)."""
    T, K = _check_gemm_args(fmt, w, xh, O, planes=1)
    nsub = K // 16 if fmt == "q6_K" else K // 32
    out = torch.empty((T, O, nsub), dtype=torch.int32, device=xh.device)
    fn = {"q4_K": load().mmq_debug_subdots_q4K, "q6_K": load().mmq_debug_subdots_q6K,
          "q5_K": load().mmq_debug_subdots_q5K, "q8_0": load().mmq_debug_subdots_q8_0}[fmt]
    with torch.cuda.device(xh.device):
        st = fn(_ptr(w), _ptr(xh), _ptr(out), T, O, K, _stream(xh.device))
    _check("mmq_debug_subdots", st)
    return out


# ---------------------------------------------- decode: around the products ---

CACHE_DTYPES = {torch.float16: 0, torch.bfloat16: 1}        # MMQ_F16, MMQ_BF16
PROB_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
ATTN_NEW_MAX = 16         # mmq_attn_decode


def _need(t, name, dtype, shape, index):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on CUDA device {index}")


class KVCache:
    """Paged key-value cache of one layer over the caller's tensors.

    k, v    float16 or bfloat16 [pages][heads][page_size][dim], unit stride along dim,
            the other strides free (multiples of 8): a transposed view of
            [pages][page_size][heads][dim] is fine;
    table   int32 [seqs][cols]: the page of every page_size entries of a sequence;
    lens    int32 [seqs]: entries of each sequence, the running step's new tokens
            included (raise it once per step, before the step's first layer);
    weight  float32 [pages][heads][page_size], attention weight received so far, or None;
    pos     int32 [pages][heads][page_size], positions of the entries, or None.

    The tensors are the state: the object keeps references and their addresses, so
    update them in place (set_bookkeeping exchanges weight and pos after kv_evict)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                 weight: torch.Tensor | None = None, pos: torch.Tensor | None = None):
        _need_cuda(k, v, table, lens, weight, pos)
        if k.dtype not in CACHE_DTYPES or k.dim() != 4 or v.dtype != k.dtype or v.shape != k.shape or v.device != k.device:
            raise ValueError("k and v must be float16 or bfloat16 [pages][heads][page_size][dim], alike")
        for t in (k, v):
            if t.stride(3) != 1 or any(s % 8 for s in t.stride()[:3]) or t.data_ptr() % 16:
                raise ValueError("k and v need unit stride along dim, the other strides multiples of 8, and 16-byte alignment")
        if table.dim() != 2 or lens.dim() != 1 or lens.shape[0] != table.shape[0]:
            raise ValueError("table must be [seqs][cols] and lens [seqs]")
        pages, heads, page_size, dim = k.shape
        seqs, cols = table.shape
        self.device, self.index = k.device, k.get_device()
        _need(table, "table", torch.int32, (seqs, cols), self.index)
        _need(lens, "lens", torch.int32, (seqs,), self.index)
        self.k, self.v, self.table, self.lens = k, v, table, lens
        self.heads, self.dim, self.page_size, self.seqs, self.cols = heads, dim, page_size, seqs, cols
        self._c = KVCacheC(_ptr(k), _ptr(v), None, None, _ptr(table), _ptr(lens), *k.stride()[:3], *v.stride()[:3], pages,
                           CACHE_DTYPES[k.dtype], heads, dim, page_size, seqs, cols)
        self._ref = ctypes.byref(self._c)
        self._work: dict = {}
        self.set_bookkeeping(weight, pos)

    def set_bookkeeping(self, weight: torch.Tensor | None, pos: torch.Tensor | None):
        """Use these weight and pos tensors from now on."""
        shape = tuple(self.k.shape[:3])
        if weight is not None:
            _need(weight, "weight", torch.float32, shape, self.index)
        if pos is not None:
            _need(pos, "pos", torch.int32, shape, self.index)
        self.weight, self.pos = weight, pos
        self._c.weight, self._c.pos = _ptr(weight), _ptr(pos)

    @classmethod
    def allocate(cls, seqs: int, cols: int, heads: int, dim: int, page_size: int = 64, dtype=torch.float16,
                 device=None, track: bool = True, share: "KVCache | None" = None) -> "KVCache":
        """A cache of its own with room for cols*page_size entries per sequence, pages in order, empty;
        with `share`, on the table and lengths of another layer's cache."""
        dev = torch.device(device if device is not None else "cuda")
        shape = (seqs * cols, heads, page_size)
        k, v = (torch.zeros(shape + (dim,), dtype=dtype, device=dev) for _ in range(2))
        if share is None:
            table = torch.arange(seqs * cols, dtype=torch.int32, device=dev).view(seqs, cols)
            lens = torch.zeros(seqs, dtype=torch.int32, device=dev)
        else:
            table, lens = share.table, share.lens
        return cls(k, v, table, lens, torch.zeros(shape, dtype=torch.float32, device=dev) if track else None,
                   torch.zeros(shape, dtype=torch.int32, device=dev) if track else None)


# The current stream's handle without the Stream object around it (2 us of every call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current = torch.cuda.current_device


class RopeTable:
    """Rotation of mmq_rope_append: freq int64 [rot/2] (turns per position as 64-bit
    fractions), rot values of each head rotated, magnitude times the result."""

    def __init__(self, freq: torch.Tensor, magnitude: float = 1.0):
        _need_cuda(freq)
        _need(freq, "freq", torch.int64, (freq.numel(),), freq.get_device())
        self.freq, self.rot, self.magnitude = freq, 2 * freq.numel(), float(magnitude)
        self.index, self.ptr = freq.get_device(), freq.data_ptr()


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, context: int = 4096,
                     fast: float = 32.0, slow: float = 1.0) -> tuple[list[float], float]:
    """(radians per position of the rot/2 pairs, magnitude), in float64.

    Pair i turns by base^(-2i/rot) per position.  scaling "linear" divides positions by
    `factor` (position interpolation).  "base" raises the base to base*factor^(rot/(rot-2)),
    which stretches the slowest pair by `factor` and leaves the fastest.  "by_parts" (YaRN,
    Peng et al. 2023) divides by `factor` the pairs that turn less than `slow` times over
    `context` positions, keeps those that turn more than `fast` times, blends linearly
    between, and scales the rotated values by 0.1 ln(factor) + 1."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if base <= 0 or factor < 1 or context < 1 or fast <= slow:
        raise ValueError("base > 0, factor >= 1, context >= 1 and fast > slow are needed")
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    inv = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling in ("none", "base"):
        return inv, 1.0
    if scaling == "linear":
        return [f / factor for f in inv], 1.0
    if scaling != "by_parts":
        raise ValueError(f"unknown scaling {scaling!r}")
    out = []
    for f in inv:
        keep = min(1.0, max(0.0, (context * f / (2 * math.pi) - slow) / (fast - slow)))
        out.append(f * keep + f / factor * (1.0 - keep))
    return out, 0.1 * math.log(factor) + 1.0


def rope_fixed(inv: list[float]) -> list[int]:
    """Radians per position as signed 64-bit fractions of a turn."""
    return [((int(f / (2 * math.pi) * 2.0 ** 64) + (1 << 63)) % (1 << 64)) - (1 << 63) for f in inv]


def rope_table(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, context: int = 4096,
               fast: float = 32.0, slow: float = 1.0, device=None) -> RopeTable:
    """The rotation table of rope_frequencies, on the device."""
    inv, magnitude = rope_frequencies(rot, base, scaling, factor, context, fast, slow)
    return RopeTable(torch.tensor(rope_fixed(inv), dtype=torch.int64).to(device if device is not None else "cuda"), magnitude)


def _rows(t, name, heads, dim, index):
    """Row stride of f32 [rows][heads][dim], shape checked, whose rows may lie apart."""
    if t.dtype is not torch.float32 or t.get_device() != index:
        raise ValueError(f"{name} must be float32 on CUDA device {index}")
    st = t.stride()
    if st[2] != 1 or (heads > 1 and st[1] != dim):
        raise ValueError(f"{name}: a row's heads must be contiguous")
    return st[0] if t.shape[0] > 1 else heads * dim          # the distance of one row from the next does not matter


def _q_shape(cache, shape):
    """(rows, query heads, new tokens per sequence) of q."""
    if len(shape) != 3 or shape[2] != cache.dim:
        raise ValueError(f"q must be [rows][q_heads][{cache.dim}]")
    if cache.seqs == 0 or shape[0] % cache.seqs:
        raise ValueError("rows must be a multiple of the cache's sequences")
    return shape[0], shape[1], shape[0] // cache.seqs


def rope_append(cache: KVCache, rope: RopeTable, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
                interleaved: bool = False, new: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotate the new tokens' q and k rows and append k and v to the cache; returns the rotated q.

    q f32 [seqs*n][q_heads][dim], k and v f32 [seqs*n][heads][dim] (rows may be slices of
    one wider product row), pos int32 [seqs*n] positions.  new int32 [seqs] limits how many
    of a sequence's n rows are there; they become the last entries of cache.lens.  `out`
    may be q."""
    index, dim, heads = cache.index, cache.dim, cache.heads
    if index != _current():
        with torch.cuda.device(index):
            return rope_append(cache, rope, q, k, v, pos, interleaved, new, out)
    shape = q.shape
    rows, q_heads, n = _q_shape(cache, shape)
    if k.shape != (rows, heads, dim) or v.shape != k.shape:
        raise ValueError(f"k and v must be [{rows}][{heads}][{dim}]")
    ldq, ldk, ldv = _rows(q, "q", q_heads, dim, index), _rows(k, "k", heads, dim, index), _rows(v, "v", heads, dim, index)
    _need(pos, "pos", torch.int32, (rows,), index)
    if new is not None:
        _need(new, "new", torch.int32, (cache.seqs,), index)
    if rope.rot > dim or rope.index != index:
        raise ValueError("the table rotates more values than a head has, or is on another device")
    stream = _raw_stream(index)
    if out is None:
        out, ldo = torch.empty(shape, dtype=torch.float32, device=cache.device), q_heads * dim
    else:
        if out.shape != shape:
            raise ValueError("out must have q's shape")
        ldo = _rows(out, "out", q_heads, dim, index)
    st = load().mmq_rope_append(cache._ref, rope.ptr, rope.rot, rope.magnitude, int(interleaved), q.data_ptr(), ldq, k.data_ptr(), ldk,
                                v.data_ptr(), ldv, pos.data_ptr(), None if new is None else new.data_ptr(), out.data_ptr(), ldo,
                                q_heads, n, stream)
    if st != 0:
        raise MMQError("mmq_rope_append", st)
    return out


class AttnWorkspace:
    """Caller-owned scratch of attn_decode: the parts of split rows (and the scores where
    weights are accumulated).  Calls that share one must be ordered (one stream)."""

    def __init__(self, device, floats: int):
        self.work = torch.empty(max(4, floats), dtype=torch.float32, device=device)
        self.floats, self.ptr, self.index = self.work.numel(), self.work.data_ptr(), self.work.get_device()

    def fits(self, floats: int) -> bool:
        return floats <= self.floats


def attn_sizes(cache: KVCache, q_heads: int, new_tokens: int = 1, accumulate: bool = False) -> int:
    """Floats of attn_decode's workspace."""
    nf = ctypes.c_int64(0)
    with torch.cuda.device(cache.device):
        st = load().mmq_attn_sizes(cache._ref, q_heads, new_tokens, int(accumulate), ctypes.byref(nf))
    _check("mmq_attn_sizes", st)
    return nf.value


def attn_workspace(cache: KVCache, q_heads: int, new_tokens: int = 1, accumulate: bool = False) -> AttnWorkspace:
    return AttnWorkspace(cache.device, attn_sizes(cache, q_heads, new_tokens, accumulate))


def attn_decode(cache: KVCache, q: torch.Tensor, scale: float | None = None, new: torch.Tensor | None = None,
                accumulate: bool = False, out: torch.Tensor | None = None,
                workspace: AttnWorkspace | None = None) -> torch.Tensor:
    """Attention of the newest n <= 16 tokens of every sequence over the cache; f32
    [seqs*n][q_heads][dim].

    q f32 [seqs*n][q_heads][dim], rotated; row t of a sequence sees the entries up to its
    own (new int32 [seqs] limits the rows as in rope_append; rows past it get 0).  scale
    defaults to dim^-0.5.  accumulate adds every entry's weight to cache.weight (no
    page may belong to two sequences then).  Drafted rows are attended without it, and those
    that stay again with it, once lens is lowered (new: how many), since a rejected row's
    weights cannot be taken back.  Without `workspace` one is allocated for this call."""
    index, dim = cache.index, cache.dim
    if index != _current():
        with torch.cuda.device(index):
            return attn_decode(cache, q, scale, new, accumulate, out, workspace)
    shape = q.shape
    key = (shape, accumulate)
    plan = cache._work.get(key)
    if plan is None:                                     # what depends on the shape alone
        rows, q_heads, n = _q_shape(cache, shape)
        if q_heads % cache.heads:
            raise ValueError("q_heads must be a multiple of the cache's heads")
        if not 1 <= n <= ATTN_NEW_MAX:
            raise ValueError(f"1 to {ATTN_NEW_MAX} new tokens per sequence")
        plan = cache._work[key] = (q_heads, n, attn_sizes(cache, q_heads, n, accumulate))
    q_heads, n, floats = plan
    ldq = _rows(q, "q", q_heads, dim, index)
    if accumulate and cache.weight is None:
        raise ValueError("the cache keeps no weights")
    if new is not None:
        _need(new, "new", torch.int32, (cache.seqs,), index)
    stream = _raw_stream(index)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=cache.device)
    else:
        _need(out, "out", torch.float32, shape, index)
    if workspace is None or not workspace.fits(floats):
        workspace = AttnWorkspace(cache.device, floats)
    elif workspace.index != index:
        raise ValueError(f"workspace must be on CUDA device {index}")
    st = load().mmq_attn_decode(cache._ref, q.data_ptr(), ldq, None if new is None else new.data_ptr(), out.data_ptr(), q_heads, n,
                                dim ** -0.5 if scale is None else scale, int(accumulate), workspace.ptr, stream)
    if st != 0:
        raise MMQError("mmq_attn_decode", st)
    return out


def _evict_ints(cache: KVCache, budget: int) -> int:
    n = ctypes.c_int64(0)
    _check("mmq_evict_sizes", load().mmq_evict_sizes(cache._ref, budget, ctypes.byref(n)))
    return n.value


def evict_workspace(cache: KVCache, budget: int) -> torch.Tensor:
    """Scratch of kv_evict (int32)."""
    return torch.empty(max(1, _evict_ints(cache, budget)), dtype=torch.int32, device=cache.device)


def kv_evict(cache: KVCache, budget: int, keep_from: torch.Tensor, weight_out: torch.Tensor, pos_out: torch.Tensor,
             workspace: torch.Tensor | None = None):
    """Cut every sequence down to `budget` entries per head: those with pos >= keep_from
    [seqs] (int32) first, then those of the largest weight.  k and v are compacted in place;
    the new bookkeeping goes to weight_out and pos_out (shaped as cache.weight), for
    cache.set_bookkeeping.  Lower cache.lens to the budget (clamp_) once every layer that
    shares it is done."""
    index, weight = cache.index, cache.weight
    if index != _current():
        with torch.cuda.device(index):
            return kv_evict(cache, budget, keep_from, weight_out, pos_out, workspace)
    if weight is None or cache.pos is None:
        raise ValueError("the cache keeps no weights or positions")
    if weight_out is None or pos_out is None:
        raise ValueError("weight_out and pos_out are required")
    shape = weight.shape
    _need(keep_from, "keep_from", torch.int32, (cache.seqs,), index)
    _need(weight_out, "weight_out", torch.float32, shape, index)
    _need(pos_out, "pos_out", torch.int32, shape, index)
    wp, pp = weight_out.data_ptr(), pos_out.data_ptr()
    if wp == weight.data_ptr() or pp == cache.pos.data_ptr():
        raise ValueError("weight_out and pos_out must not be the cache's own")
    need = cache._work.get(budget)
    if need is None:
        need = cache._work[budget] = _evict_ints(cache, budget)
    if workspace is None:
        workspace = torch.empty(max(1, need), dtype=torch.int32, device=cache.device)
    elif workspace.dtype is not torch.int32 or workspace.get_device() != index or not workspace.is_contiguous() or workspace.numel() < need:
        raise ValueError("workspace must be evict_workspace(cache, budget) or larger")
    st = load().mmq_kv_evict(cache._ref, budget, keep_from.data_ptr(), wp, pp, workspace.data_ptr(), _raw_stream(index))
    if st != 0:
        raise MMQError("mmq_kv_evict", st)


def spec_verify(target: torch.Tensor, draft: torch.Tensor | None, tokens: torch.Tensor, uniform: torch.Tensor,
                count: torch.Tensor | None = None, out=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Verify drafted tokens against the target's probabilities (speculative sampling).

    target [seqs][n+1][vocab] and draft [seqs][n][vocab] probabilities (f32, f16 or bf16,
    alike; draft None: the drafts were not sampled), tokens int32 [seqs][n], uniform f32
    [seqs][n+1] in [0, 1), count int32 [seqs] drafts there (None: n).  Returns (tokens
    int32 [seqs][n+1]: the accepted ones, one drawn, then -1; accepted int32 [seqs]);
    `out` may supply the two."""
    dtype, index = PROB_DTYPES.get(target.dtype), target.get_device()
    shape = target.shape
    if dtype is None or index < 0 or len(shape) != 3 or shape[1] < 2 or not target.is_contiguous():
        raise ValueError("target must be a contiguous CUDA tensor [seqs][drafts+1][vocab] of probabilities")
    if index != _current():
        with torch.cuda.device(index):
            return spec_verify(target, draft, tokens, uniform, count, out)
    B, n1, V = shape
    if draft is not None:
        _need(draft, "draft", target.dtype, (B, n1 - 1, V), index)
    _need(tokens, "tokens", torch.int32, (B, n1 - 1), index)
    _need(uniform, "uniform", torch.float32, (B, n1), index)
    if count is not None:
        _need(count, "count", torch.int32, (B,), index)
    stream = _raw_stream(index)
    if out is None:
        dev = target.device
        res, acc = torch.empty((B, n1), dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev)
    else:
        res, acc = out
        _need(res, "out[0]", torch.int32, (B, n1), index)
        _need(acc, "out[1]", torch.int32, (B,), index)
    st = load().mmq_spec_verify(target.data_ptr(), None if draft is None else draft.data_ptr(), dtype, tokens.data_ptr(),
                                uniform.data_ptr(), None if count is None else count.data_ptr(), res.data_ptr(), acc.data_ptr(),
                                B, n1 - 1, V, stream)
    if st != 0:
        raise MMQError("mmq_spec_verify", st)
    return res, acc


# MMQ_ERR_INDEX: kernel ids and sites of csrc/mmq_cache.cuh
_INDEX_KERNELS = {32: "rotary append", 33: "attention", 34: "eviction", 35: "verification"}
_INDEX_SITES = {1: "a sequence's length", 2: "a page id", 3: "a count of new or drafted tokens", 4: "a drafted token"}
_ERR_CUDA, _ERR_INDEX = -8, -11


def _failure(st: int, detail, info) -> str:
    """What mmq_check_status reported, in words."""
    if st == _ERR_INDEX:
        return f"{_INDEX_KERNELS.get(detail[1], detail[1])}: {_INDEX_SITES.get(detail[2], detail[2])} (block {detail[3]})"
    return (f"kernel (id {detail[1]}, site {detail[2]}, block {detail[3]}; waited {info[0]} us over "
            f"{info[1]} polls for parity {info[2]} of the barrier at shared address {info[3]})")


def check_status(device: torch.device | None = None):
    """Synchronise the current stream and raise if a kernel reported an error.

    The products and the decode-side operators have a status word each; where both hold an
    error, the one raised has the products' status and names both."""
    dev = device or torch.device("cuda", torch.cuda.current_device())
    first, what = 0, []
    with torch.cuda.device(dev):
        for _ in range(2):                       # mmq_check_status clears what it reports
            detail, info = (ctypes.c_int * 4)(), (ctypes.c_int * 4)()
            st = load().mmq_check_status(_stream(dev), detail)
            if st == 0:
                break
            load().mmq_last_failure_info(info)
            what.append(_failure(st, detail, info))
            first = first or st
            if st == _ERR_CUDA:
                break
    if first != 0:
        raise MMQError("; ".join(what), first)


def tensor_peak_tmacs(kind: str = "int8", device: torch.device | None = None) -> float:
    """Measured warp-level tensor throughput (TMAC/s) of the device: 'int8' or 'f16'."""
    dev = device or torch.device("cuda", torch.cuda.current_device())
    v = ctypes.c_double(0.0)
    with torch.cuda.device(dev):
        st = load().mmq_probe_tensor_peak(0 if kind == "int8" else 1, ctypes.byref(v), _stream(dev))
    _check("mmq_probe_tensor_peak", st)
    return v.value


def mmq_forward(fmt: str, w: torch.Tensor, x: torch.Tensor, O: int) -> torch.Tensor:
    """Quantise x [T][K] to q8_1 and run the production GEMM: the whole hot path."""
    _, ds, _, xa = quantize_q8_1(x, want_qs=False, want_xh=False, want_xa=True)
    return gemm(fmt, w, xa, ds, O)
