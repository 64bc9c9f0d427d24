"""Python binding of libgqa_attn.so (include/gqa_attn.h).

Argument marshalling only: every function here takes torch tensors that already
live on the GPU, checks their dtype, shape and contiguity, and passes raw
pointers, sizes and the current CUDA stream to the C entry point of the same
name. All arithmetic runs in the library's CUDA kernels; there is no fallback.
If the shared library is missing, ``load()`` raises.
"""
import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgqa_attn.so")

F32, BF16 = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "CUDA error",
          4: "workspace missing or too small", 5: "device saw an index or length out of range",
          6: "a bounded device wait gave up"}
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE, ERR_DEVICE_BOUNDS, ERR_DEVICE_TIMEOUT = range(7)

EXPORTS = ("attn_prefill_causal", "attn_decode_contig", "attn_decode_paged", "kv_append_paged",
           "attn_rope_interleaved", "attn_decode_workspace_bytes", "attn_get_device_error",
           "gqa_status_string", "gqa_debug_withhold_first_tile", "attn_decode_paged_static_workspace",
           "attn_prefill_causal_ex", "attn_decode_contig_ex", "attn_decode_paged_ex", "attn_prefill_paged",
           "attn_prefill_paged_ex", "mla_absorb_q", "attn_decode_mla_absorbed",
           "attn_decode_mla_absorbed_workspace_bytes", "mla_unabsorb_out", "attn_decode_mla_absorbed_paged",
           "attn_rope_interleaved_qk", "gqa_rope_frequencies", "attn_qk_norm_rope", "kv_append_paged_rows",
           "attn_decode_shared_prefix", "attn_decode_shared_prefix_workspace_bytes", "attn_cross",
           "attn_cross_workspace_bytes", "kv_plan_rows", "kv_append_slots", "kv_commit_rows",
           "attn_tree_paged", "attn_tree_paged_workspace_bytes")


class GqaArms(ctypes.Structure):
    """`gqa_arms` (include/gqa_attn.h): window, softcap, sinks, ALiBi slopes."""
    _fields_ = [("window", ctypes.c_int), ("softcap", ctypes.c_float), ("sinks", ctypes.c_void_p),
                ("alibi_slopes", ctypes.c_void_p)]


class GqaHeads(ctypes.Structure):
    """`gqa_heads` (include/gqa_attn.h): a strided tensor [batch, tokens, heads, d]."""
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class GqaRopeScaling(ctypes.Structure):
    """`gqa_rope_scaling` (include/gqa_attn.h)."""
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_double), ("original_max", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("magnitude", ctypes.c_double),
                ("divisors", ctypes.c_void_p)]


class GqaRope(ctypes.Structure):
    """`gqa_rope` (include/gqa_attn.h); made by rope_init, which keeps the device
    copy of the frequencies in `table`."""
    _fields_ = [("layout", ctypes.c_int), ("rot_offset", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("magnitude", ctypes.c_float), ("freqs", ctypes.c_void_p)]


ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "turns": 2, "index": 3}

STATIC_WORKSPACE_BYTES = 16 << 20  # GQA_STATIC_WORKSPACE_BYTES

_lib = None


class GqaError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status})")


def load(path: str = None):
    """Load the shared library (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, I, F, D, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_double, ctypes.c_size_t
    sig = {
        "attn_prefill_causal": [P, P, P, P, I, I, I, P, I, I, I, I, F, I, P],
        "attn_decode_contig": [P, P, P, P, I, P, P, I, I, I, I, I, I, F, I, P, S, P],
        "attn_decode_paged": [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, P, S, P],
        "attn_decode_paged_static_workspace": [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, P],
        "kv_append_paged": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, D, I, I, I, P],
        "attn_rope_interleaved": [P, P, I, I, I, I, I, I, I, D, I, P],
        "attn_rope_interleaved_qk": [P, P, P, I, I, I, I, I, I, I, I, I, D, I, P],
        "attn_get_device_error": [P],
        "attn_prefill_causal_ex": [P, P, P, P, I, I, I, P, I, I, I, I, F, I, P, P],
        "attn_decode_contig_ex": [P, P, P, P, I, P, P, I, I, I, I, I, I, F, I, P, S, P, P],
        "attn_decode_paged_ex": [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, P, S, P, P],
        "attn_prefill_paged": [P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, P],
        "attn_prefill_paged_ex": [P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, P, P],
        "gqa_debug_withhold_first_tile": [I],
        "mla_absorb_q": [P, P, P, I, I, I, I, I, I, P],
        "attn_decode_mla_absorbed": [P, P, P, P, I, I, I, I, I, F, I, P, S, P],
        "mla_unabsorb_out": [P, P, P, I, I, I, I, I, P],
        "attn_decode_mla_absorbed_paged": [P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, S, P],
        "attn_decode_shared_prefix": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, P, S, P, P],
        "attn_cross": [P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, S, P],
        "gqa_rope_frequencies": [P, P, I, D, P],
        "attn_qk_norm_rope": [P, P, P, P, P, P, F, P, I, I, I, I, I, P, I, P],
        "kv_append_paged_rows": [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, P, P, F, P, I, P],
        "kv_plan_rows": [P] * 14 + [I] * 6 + [P],
        "kv_append_slots": [P] * 8 + [I] * 7 + [P, P, F, P, I, P],
        "attn_tree_paged": [P] * 8 + [I] * 11 + [F, I, P, S, P, P],
        "kv_commit_rows": [P, P, I] + [P] * 6 + [I] * 8 + [I, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.attn_decode_workspace_bytes.argtypes = [I, I, I, I]
    lib.attn_decode_workspace_bytes.restype = S
    lib.attn_decode_mla_absorbed_workspace_bytes.argtypes = [I, I, I, I]
    lib.attn_decode_mla_absorbed_workspace_bytes.restype = S
    lib.attn_decode_shared_prefix_workspace_bytes.argtypes = [I] * 6
    lib.attn_decode_shared_prefix_workspace_bytes.restype = S
    lib.attn_cross_workspace_bytes.argtypes = [I] * 8
    lib.attn_cross_workspace_bytes.restype = S
    lib.attn_tree_paged_workspace_bytes.argtypes = [I] * 9
    lib.attn_tree_paged_workspace_bytes.restype = S
    lib.gqa_status_string.argtypes = [I]
    lib.gqa_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _dtype(*ts):
    dts = {t.dtype for t in ts if t is not None}
    if len(dts) != 1:
        raise TypeError(f"tensors must share one dtype, got {dts}")
    dt = dts.pop()
    if dt == torch.bfloat16:
        return BF16
    if dt == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {dt}")


def _p(t):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


def _i32(t):
    if t is not None and t.dtype != torch.int32:
        raise TypeError("index tensors must be int32")
    return _p(t)


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    # the handle of torch.cuda.current_stream() without building a Stream object for
    # it, which took 3 us of a call's 14 on a Grace core
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


def _check(status, what):
    if status != OK:
        raise GqaError(status, what)


def _arms(window, softcap, sinks, alibi_slopes):
    """The `gqa_arms` struct (by reference), or None when every arm is off."""
    if not window and not softcap and sinks is None and alibi_slopes is None:
        return None
    for t in (sinks, alibi_slopes):
        if t is not None and t.dtype != torch.float32:
            raise TypeError("sinks and alibi_slopes must be float32 [H]")
    return ctypes.byref(GqaArms(int(window or 0), float(softcap or 0.0), _p(sinks), _p(alibi_slopes)))


def attn_prefill_causal(q, k, v, out, attention_scale, position_offset=None, stream=None, window=0, softcap=0.0,
                        sinks=None, alibi_slopes=None):
    """q [B, S, H, dk], k [B, Hkv, S_kv, dk], v [B, Hkv, S_kv, dv], out [B, S, H, dv].
    window / softcap / sinks / alibi_slopes: the arms (include/gqa_attn.h, `gqa_arms`)."""
    B, S, H, dk = q.shape
    _, Hkv, S_kv, dv = v.shape
    arms = _arms(window, softcap, sinks, alibi_slopes)
    args = (_p(q), _p(k), _p(v), _p(out), B, S, S_kv, _i32(position_offset), H, Hkv, dk, dv, float(attention_scale),
            _dtype(q, k, v, out))
    if arms is None:
        _check(load().attn_prefill_causal(*args, _stream(stream)), "attn_prefill_causal")
    else:
        _check(load().attn_prefill_causal_ex(*args, arms, _stream(stream)), "attn_prefill_causal_ex")
    return out


def attn_prefill_paged(q, k_pool, v_pool, block_tables, out, attention_scale, position_offset=None, stream=None,
                       window=0, softcap=0.0, sinks=None, alibi_slopes=None):
    """Chunked prefill against the paged pool: q [B, S, H, dk]; pools [num_blocks, Hkv, bs, d];
    block_tables int32 [B, mbps]; position_offset int32 [B] or None; out [B, S, H, dv].
    window / softcap / sinks / alibi_slopes: the arms (`gqa_arms`)."""
    B, S, H, dk = q.shape
    nb, Hkv, bs, dv = v_pool.shape
    arms = _arms(window, softcap, sinks, alibi_slopes)
    args = (_p(q), _p(k_pool), _p(v_pool), _i32(block_tables), _i32(position_offset), _p(out), B, S,
            block_tables.shape[1], nb, bs, H, Hkv, dk, dv, float(attention_scale), _dtype(q, k_pool, v_pool, out))
    if arms is None:
        _check(load().attn_prefill_paged(*args, _stream(stream)), "attn_prefill_paged")
    else:
        _check(load().attn_prefill_paged_ex(*args, arms, _stream(stream)), "attn_prefill_paged_ex")
    return out


def attn_decode_workspace_bytes(B, H, d_v, max_len):
    return int(load().attn_decode_workspace_bytes(B, H, d_v, max_len))


def decode_workspace(B, H, d_v, max_len, device="cuda"):
    """A workspace tensor of the size the decode calls need (None when none)."""
    n = attn_decode_workspace_bytes(B, H, d_v, max_len)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def attn_decode_contig(q, k_cache, v_cache, seq_lens, out, attention_scale, workspace=None, k_rot_shared=None,
                       stream=None, window=0, softcap=0.0, sinks=None, alibi_slopes=None):
    """q [B, H, dk]; k_cache [B, Hkv, L, dk - d_rot]; v_cache [B, Hkv, L, dv];
    k_rot_shared None or [B, L, d_rot]; seq_lens int32 [B]; out [B, H, dv];
    window / softcap / sinks / alibi_slopes: the arms (`gqa_arms`)."""
    B, H, dk = q.shape
    _, Hkv, L, dv = v_cache.shape
    d_rot = 0 if k_rot_shared is None else k_rot_shared.shape[-1]
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    arms = _arms(window, softcap, sinks, alibi_slopes)
    args = (_p(q), _p(k_cache), _p(v_cache), _p(k_rot_shared), d_rot, _i32(seq_lens), _p(out), B, L, H, Hkv, dk, dv,
            float(attention_scale), _dtype(q, k_cache, v_cache, out, k_rot_shared), _p(workspace), ws)
    if arms is None:
        _check(load().attn_decode_contig(*args, _stream(stream)), "attn_decode_contig")
    else:
        _check(load().attn_decode_contig_ex(*args, arms, _stream(stream)), "attn_decode_contig_ex")
    return out


def attn_decode_paged(q, k_pool, v_pool, block_tables, seq_lens, out, attention_scale, workspace=None,
                      stream=None, window=0, softcap=0.0, sinks=None, alibi_slopes=None):
    """q [B, H, dk]; pools [num_blocks, Hkv, bs, d]; block_tables int32 [B, mbps];
    window / softcap / sinks / alibi_slopes: the arms (`gqa_arms`)."""
    B, H, dk = q.shape
    nb, Hkv, bs, dv = v_pool.shape
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    arms = _arms(window, softcap, sinks, alibi_slopes)
    args = (_p(q), _p(k_pool), _p(v_pool), _i32(block_tables), _i32(seq_lens), _p(out), B, block_tables.shape[1], nb,
            bs, H, Hkv, dk, dv, float(attention_scale), _dtype(q, k_pool, v_pool, out), _p(workspace), ws)
    if arms is None:
        _check(load().attn_decode_paged(*args, _stream(stream)), "attn_decode_paged")
    else:
        _check(load().attn_decode_paged_ex(*args, arms, _stream(stream)), "attn_decode_paged_ex")
    return out


def attn_decode_paged_static_workspace(q, k_pool, v_pool, block_tables, seq_lens, out, attention_scale,
                                       stream=None):
    """attn_decode_paged with the library's fixed device scratch instead of a
    caller-allocated workspace (for callers that cannot allocate device memory;
    see include/gqa_attn.h). Raises GqaError(ERR_WORKSPACE) when the problem needs
    more than STATIC_WORKSPACE_BYTES of scratch."""
    B, H, dk = q.shape
    nb, Hkv, bs, dv = v_pool.shape
    _check(load().attn_decode_paged_static_workspace(_p(q), _p(k_pool), _p(v_pool), _i32(block_tables),
                                                     _i32(seq_lens), _p(out), B, block_tables.shape[1], nb, bs, H,
                                                     Hkv, dk, dv, float(attention_scale),
                                                     _dtype(q, k_pool, v_pool, out), _stream(stream)),
           "attn_decode_paged_static_workspace")
    return out


def mla_absorb_q(q, k_b, q_abs, stream=None):
    """q [B, H, d_nope + d_rope]; k_b [H, d_c, d_nope]; q_abs [B, H, d_c + d_rope] (bf16)."""
    B, H, dq = q.shape
    _, d_c, d_nope = k_b.shape
    _check(load().mla_absorb_q(_p(q), _p(k_b), _p(q_abs), B, H, d_nope, dq - d_nope, d_c, _dtype(q, k_b, q_abs),
                               _stream(stream)), "mla_absorb_q")
    return q_abs


def attn_decode_mla_absorbed_workspace_bytes(B, H, d_c, max_len):
    return int(load().attn_decode_mla_absorbed_workspace_bytes(B, H, d_c, max_len))


def mla_absorbed_workspace(B, H, d_c, max_len, device="cuda"):
    """A workspace tensor of the size attn_decode_mla_absorbed needs (None when none)."""
    n = attn_decode_mla_absorbed_workspace_bytes(B, H, d_c, max_len)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def attn_decode_mla_absorbed(q_abs, latent, seq_lens, out_lat, attention_scale, workspace=None, stream=None):
    """q_abs [B, H, d_c + d_r]; latent [B, L, d_c + d_r]; seq_lens int32 [B];
    out_lat [B, H, d_c] (bf16)."""
    B, H, w = q_abs.shape
    _, L, _ = latent.shape
    d_c = out_lat.shape[-1]
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().attn_decode_mla_absorbed(_p(q_abs), _p(latent), _i32(seq_lens), _p(out_lat), B, L, H, d_c, w - d_c,
                                           float(attention_scale), _dtype(q_abs, latent, out_lat), _p(workspace), ws,
                                           _stream(stream)), "attn_decode_mla_absorbed")
    return out_lat


def attn_decode_mla_absorbed_paged(q_abs, latent_pool, block_tables, seq_lens, out_lat, attention_scale,
                                   workspace=None, stream=None):
    """q_abs [B, H, d_c + d_r]; latent_pool [num_blocks, bs, d_c + d_r]; block_tables int32
    [B, mbps]; seq_lens int32 [B]; out_lat [B, H, d_c] (bf16)."""
    B, H, w = q_abs.shape
    nb, bs, _ = latent_pool.shape
    d_c = out_lat.shape[-1]
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().attn_decode_mla_absorbed_paged(_p(q_abs), _p(latent_pool), _i32(block_tables), _i32(seq_lens),
                                                 _p(out_lat), B, block_tables.shape[1], nb, bs, H, d_c, w - d_c,
                                                 float(attention_scale), _dtype(q_abs, latent_pool, out_lat),
                                                 _p(workspace), ws, _stream(stream)),
           "attn_decode_mla_absorbed_paged")
    return out_lat


def mla_unabsorb_out(out_lat, v_b, out, stream=None):
    """out_lat [B, H, d_c]; v_b [H, d_v, d_c]; out [B, H, d_v] (bf16)."""
    B, H, d_c = out_lat.shape
    d_v = v_b.shape[1]
    _check(load().mla_unabsorb_out(_p(out_lat), _p(v_b), _p(out), B, H, d_c, d_v, _dtype(out_lat, v_b, out),
                                   _stream(stream)), "mla_unabsorb_out")
    return out


def kv_append_paged(q, k_new, v_new, k_pool, v_pool, block_tables, seq_lens_in, seq_lens_out, rope_theta,
                    rot_offset=0, rot_dim=None, stream=None):
    """Rotate q and k_new at p = seq_lens_in[b], write k/v into the pools, set
    seq_lens_out = p + 1 (may be the same tensor as seq_lens_in)."""
    B, H, dk = q.shape
    nb, Hkv, bs, dv = v_pool.shape
    rot_dim = dk - rot_offset if rot_dim is None else rot_dim
    _check(load().kv_append_paged(_p(q), _p(k_new), _p(v_new), _p(k_pool), _p(v_pool), _i32(block_tables),
                                  _i32(seq_lens_in), _i32(seq_lens_out), B, block_tables.shape[1], nb, bs, H,
                                  Hkv, dk, dv, float(rope_theta), rot_offset, rot_dim,
                                  _dtype(q, k_new, v_new, k_pool, v_pool), _stream(stream)), "kv_append_paged")


def attn_rope_interleaved(x, positions, theta, rot_offset=0, rot_dim=None, heads_outer=False, stream=None):
    """In place. x [B, T, heads, d] (or [B, heads, T, d] with heads_outer); positions int32 [B, T]."""
    if heads_outer:
        B, heads, T, d = x.shape
    else:
        B, T, heads, d = x.shape
    rot_dim = d - rot_offset if rot_dim is None else rot_dim
    _check(load().attn_rope_interleaved(_p(x), _i32(positions), B, T, heads, d, int(bool(heads_outer)),
                                        rot_offset, rot_dim, float(theta), _dtype(x), _stream(stream)),
           "attn_rope_interleaved")
    return x


def attn_rope_interleaved_qk(q, k, positions, theta, rot_offset=0, rot_dim=None, q_heads_outer=False,
                             k_heads_outer=False, stream=None):
    """In place, one launch. q [B, T, heads_q, d] (or [B, heads_q, T, d] with
    q_heads_outer), k likewise; positions int32 [B, T]."""
    if q_heads_outer:
        B, hq, T, d = q.shape
    else:
        B, T, hq, d = q.shape
    hk = k.shape[1] if k_heads_outer else k.shape[2]
    rot_dim = d - rot_offset if rot_dim is None else rot_dim
    _check(load().attn_rope_interleaved_qk(_p(q), _p(k), _i32(positions), B, T, hq, hk, d, int(bool(q_heads_outer)),
                                           int(bool(k_heads_outer)), rot_offset, rot_dim, float(theta), _dtype(q),
                                           _stream(stream)), "attn_rope_interleaved_qk")
    return q, k


def _here(*ts):
    """Check that the tensors live on the current CUDA device (calls launch there)."""
    dev = torch.cuda.current_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors must live on the current CUDA device")


_pack_view = struct.Struct("4q").pack  # `gqa_heads`, which a call only reads


def _view(t, ndim):
    """The bytes of `gqa_heads` of a [B, T, heads, d] (ndim 4) or [N, heads, d] (ndim 3)
    tensor with a dense last axis and any other strides; None stays None."""
    if t is None:
        return None
    st = t.stride()
    if len(st) != ndim:
        raise ValueError(f"expected {ndim} axes, got shape {tuple(t.shape)}")
    if st[-1] != 1:
        raise ValueError("the last axis must be dense")
    return _pack_view(t.data_ptr(), *st[:3]) if ndim == 4 else _pack_view(t.data_ptr(), 0, st[0], st[1])


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _writes_once(*ts):
    for t in ts:
        if t is not None and 0 in t.stride() and any(s == 0 and n > 1 for s, n in zip(t.stride(), t.shape)):
            raise ValueError("an output must not be broadcast")


def _weight(w, d):
    if w is not None and w.shape != (d,):
        raise ValueError(f"a norm weight must be [{d}], got {tuple(w.shape)}")
    return _p(w)


def attn_decode_shared_prefix_workspace_bytes(B, H, Hkv, d_v, max_len, n_groups):
    return int(load().attn_decode_shared_prefix_workspace_bytes(B, H, Hkv, d_v, max_len, n_groups))


def shared_prefix_workspace(B, H, Hkv, d_v, max_len, n_groups, device="cuda"):
    """A workspace tensor of the size attn_decode_shared_prefix needs (max_len: rows a table row can name)."""
    n = attn_decode_shared_prefix_workspace_bytes(B, H, Hkv, d_v, max_len, n_groups)
    return torch.empty(n, dtype=torch.uint8, device=device)


def attn_decode_shared_prefix(q, k_pool, v_pool, block_tables, seq_lens, group_starts, shared_blocks, out,
                              attention_scale, workspace, stream=None, window=0, softcap=0.0, sinks=None,
                              alibi_slopes=None):
    """attn_decode_paged for a batch in groups: sequences group_starts[g] .. group_starts[g + 1] - 1
    (int32 [n_groups + 1]) share their tables' first shared_blocks[g] (int32 [n_groups]) blocks, whose
    rows are read once a group. q [B, H, dk]; pools [num_blocks, Hkv, bs, d]; block_tables int32
    [B, mbps]; workspace from shared_prefix_workspace; window / softcap / sinks / alibi_slopes: the arms."""
    B, H, dk = q.shape
    nb, Hkv, bs, dv = v_pool.shape
    n = shared_blocks.shape[0]
    if (k_pool.shape != (nb, Hkv, bs, dk) or out.shape != (B, H, dv) or block_tables.shape[0] != B or
            seq_lens.numel() != B or group_starts.numel() != n + 1):
        raise ValueError("q, the pools, the tables, the lengths, the groups and out do not agree")
    _here(q, k_pool, v_pool, block_tables, seq_lens, group_starts, shared_blocks, out, workspace, sinks, alibi_slopes)
    if any(x is not None and x.numel() != H for x in (sinks, alibi_slopes)):
        raise ValueError("sinks and alibi_slopes must be float32 [H]")
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().attn_decode_shared_prefix(
        _p(q), _p(k_pool), _p(v_pool), _i32(block_tables), _i32(seq_lens), _i32(group_starts), _i32(shared_blocks),
        _p(out), B, n, block_tables.shape[1], nb, bs, H, Hkv, dk, dv, float(attention_scale),
        _dtype(q, k_pool, v_pool, out), _p(workspace), ws, _arms(window, softcap, sinks, alibi_slopes),
        _stream(stream)), "attn_decode_shared_prefix")
    return out


def attn_cross_workspace_bytes(B, seq_q, seq_kv_max, H, Hkv, d_k, d_v, dtype=torch.bfloat16):
    return int(load().attn_cross_workspace_bytes(B, seq_q, seq_kv_max, H, Hkv, d_k, d_v,
                                                 BF16 if dtype == torch.bfloat16 else F32))


def cross_workspace(B, seq_q, H, Hkv, d_k, d_v, seq_kv_max, dtype=torch.bfloat16, device="cuda"):
    """A workspace tensor of the size attn_cross needs (None when none); it does for any smaller B and
    seq_kv_max too, not for another seq_q."""
    n = attn_cross_workspace_bytes(B, seq_q, seq_kv_max, H, Hkv, d_k, d_v, dtype)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def attn_cross(q, k, v, out, attention_scale, kv_lens=None, workspace=None, stream=None):
    """Every row sees all keys of its sequence: q [B, S, H, dk], k [B, Hkv, L, dk], v [B, Hkv, L, dv],
    out [B, S, H, dv]; kv_lens int32 [B] (None: L; a sequence of 0 keys gets zeros); workspace from
    cross_workspace."""
    B, S, H, dk = q.shape
    _, Hkv, L, dv = v.shape
    if (k.shape != (B, Hkv, L, dk) or v.shape[0] != B or out.shape != (B, S, H, dv) or
            (kv_lens is not None and kv_lens.numel() != B)):
        raise ValueError("q, k, v, kv_lens and out do not agree")
    _here(q, k, v, out, kv_lens, workspace)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().attn_cross(_p(q), _p(k), _p(v), _i32(kv_lens), _p(out), B, S, L, H, Hkv, dk, dv,
                             float(attention_scale), _dtype(q, k, v, out), _p(workspace), ws, _stream(stream)),
           "attn_cross")
    return out


def rope_frequencies(rot_dim, theta, scaling="none", factor=1.0, original_max=0.0, low=1.0, high=4.0, magnitude=0.0,
                     divisors=None):
    """The frequencies of a rotation as (host float32 tensor [rot_dim / 2, 2], magnitude);
    include/gqa_attn.h, `gqa_rope_scaling`, has the formulas. divisors: rot_dim / 2 numbers or None."""
    div = None
    if divisors is not None:
        div = (ctypes.c_double * len(divisors))(*[float(x) for x in divisors])
        if len(divisors) != rot_dim // 2:
            raise ValueError(f"divisors must have {rot_dim // 2} entries")
    sc = GqaRopeScaling(ROPE_SCALINGS[scaling], float(factor), float(original_max), float(low), float(high),
                        float(magnitude), ctypes.cast(div, ctypes.c_void_p) if div is not None else None)
    out = (ctypes.c_float * max(2, int(rot_dim)))()
    mag = ctypes.c_float()
    _check(load().gqa_rope_frequencies(out, ctypes.byref(mag), int(rot_dim), float(theta), ctypes.byref(sc)),
           "gqa_rope_frequencies")
    return torch.tensor(list(out), dtype=torch.float32).view(-1, 2), mag.value


def rope_init(rot_dim, theta, layout="interleaved", rot_offset=0, device="cuda", **scaling):
    """A rotation for attn_qk_norm_rope and kv_append_paged_rows, made once for a
    model: layout "interleaved" (adjacent pairs) or "half"; **scaling as for
    rope_frequencies. The frequencies go to `device`."""
    freqs, mag = rope_frequencies(rot_dim, theta, **scaling)
    table = freqs.to(device)
    r = GqaRope(ROPE_LAYOUTS[layout], int(rot_offset), int(rot_dim), mag, table.data_ptr())
    r.table = table
    return r


def attn_qk_norm_rope(q, k, q_out, k_out, positions, rope=None, q_weight=None, k_weight=None, eps=1e-6, stream=None):
    """RMS norm per head (a weight of None: no norm), then the rotation (rope of None:
    none). q, q_out [B, T, H, d] and k, k_out [B, T, Hkv, d], of any strides with a dense
    last axis (a head-major cache [B, Hkv, T, d] goes in as k_out.transpose(1, 2)); q with
    q_out, or k with k_out, may be None. positions int32 [B, T]. Outputs may be the inputs."""
    if q is None and k is None:
        raise ValueError("neither queries nor keys given")
    H = Hkv = 0
    if q is not None:
        B, T, H, d = q.shape
    if k is not None:
        kB, kT, Hkv, kd = k.shape
        if q is None:
            B, T, d = kB, kT, kd
        elif (kB, kT, kd) != (B, T, d):
            raise ValueError("q and k must agree in batch, tokens and width")
    if (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("an input and its output go together")
    if (q is not None and q_out.shape != q.shape) or (k is not None and k_out.shape != k.shape):
        raise ValueError("an output must have its input's shape")
    _here(q, k, q_out, k_out, positions, q_weight, k_weight, rope.table if rope is not None else None)
    _writes_once(q_out, k_out)
    if positions is not None and positions.numel() != B * T:
        raise ValueError("positions must be [B, T]")
    _check(load().attn_qk_norm_rope(
        _view(q, 4), _view(k, 4), _view(q_out, 4), _view(k_out, 4), _weight(q_weight, d), _weight(k_weight, d),
        float(eps), _i32(positions), B, T, H, Hkv, d, _ref(rope), _dtype(q, k, q_out, k_out, q_weight, k_weight),
        _stream(stream)), "attn_qk_norm_rope")
    return q_out, k_out


def kv_append_paged_rows(q, k_new, v_new, q_out, k_pool, v_pool, block_tables, row_starts, seq_lens_in, seq_lens_out,
                         rope=None, q_weight=None, k_weight=None, eps=1e-6, stream=None):
    """Norm and rotate the packed new rows q [N, H, dk] (into q_out; both may be None) and
    k_new [N, Hkv, dk], and write k_new and v_new [N, Hkv, dv] to the pools: rows
    row_starts[b] .. row_starts[b + 1] - 1 (int32 [B + 1]) go behind the seq_lens_in[b]
    rows of sequence b; seq_lens_out[b] = seq_lens_in[b] + their number (may be the same
    tensor). Inputs of any strides with a dense last axis."""
    N, Hkv, dk = k_new.shape
    nb, _, bs, dv = v_pool.shape
    B, mbps = block_tables.shape
    H = 0
    if v_new.shape != (N, Hkv, dv) or k_pool.shape != (nb, Hkv, bs, dk) or v_pool.shape[1] != Hkv:
        raise ValueError("k_new, v_new and the pools do not agree")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        H = q.shape[1]
        if q.shape != (N, H, dk) or q_out.shape != (N, H, dk):
            raise ValueError("q and q_out must both be [N, H, dk]")
    if row_starts.numel() != B + 1 or seq_lens_in.numel() != B or seq_lens_out.numel() != B:
        raise ValueError("row_starts, the lengths and block_tables do not agree in the number of sequences")
    _here(q, k_new, v_new, q_out, k_pool, v_pool, block_tables, row_starts, seq_lens_in, seq_lens_out, q_weight,
          k_weight, rope.table if rope is not None else None)
    _writes_once(q_out)
    _check(load().kv_append_paged_rows(
        _view(q, 3), _view(k_new, 3), _view(v_new, 3), _view(q_out, 3), _p(k_pool), _p(v_pool), _i32(block_tables),
        _i32(row_starts), _i32(seq_lens_in), _i32(seq_lens_out), N, B, mbps, nb, bs, H, Hkv, dk, dv,
        _weight(q_weight, dk), _weight(k_weight, dk), float(eps), _ref(rope),
        _dtype(q, k_new, v_new, q_out, k_pool, v_pool, q_weight, k_weight), _stream(stream)), "kv_append_paged_rows")
    return q_out


# The calls of a step that verifies drafted tokens take ten tensors and more, and the small ones last 3 to 12 us on
# the GPU: their arguments are looked at once each, and go as plain numbers (with the helpers above, which build an
# object for each pointer, kv_plan_rows took 12 us of a Grace core).
_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
# (absent from a build of PyTorch without CUDA, where the package can still be imported)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# torch.cuda.current_device without its look at the set-up, which the tensors show
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _at(t, dev, dtype):
    """The address of a contiguous tensor of the given type on device `dev`; None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"expected a tensor of {dtype}, got {t.dtype}")
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("tensors must be contiguous and live on the current CUDA device")
    return t.data_ptr()


def _number(dtype):
    if dtype is _BF16:
        return BF16
    if dtype is _F32:
        return F32
    raise TypeError(f"unsupported dtype {dtype}")


def kv_plan_rows(seq_lens, new_rows, block_tables, blocks_in, blocks_out, free_list, free_in, free_out, row_starts, positions,
                 slots, block_size, keep_blocks=None, parents=None, tree_mask=None, stream=None):
    """The index arrays of a step that adds new_rows[b] rows to the seq_lens[b] of sequence b (int32 [B]):
    grows block_tables int32 [B, mbps] from free_list (int32 [num_blocks], a stack of free_in[0] blocks) and
    gives back what is no longer needed; blocks_in / blocks_out int32 [B] are the entries in use before and
    after (keep_blocks of them never given back), free_out int32 [2] the blocks free afterwards and those that
    were wanting. Writes row_starts int32 [B + 1], positions int32 [N] and slots int64 [N] (-1: none). With
    parents int32 [N] (-1: the history) positions go by depth, and tree_mask int64 [N, words] gets each row's
    bits for itself and its ancestors. A sequence for which there are too few blocks keeps what it has, its rows have no
    slot and the entries that it wanted are -1. blocks_out and free_out may be blocks_in and free_in."""
    B, mbps = block_tables.shape
    N = positions.shape[0]
    words = 0
    if (parents is None) != (tree_mask is None):
        raise ValueError("parents and tree_mask go together")
    if parents is not None:
        if tree_mask.dim() != 2 or tree_mask.shape[0] != N or parents.numel() != N:
            raise ValueError("parents must be [N] and tree_mask [N, words]")
        words = tree_mask.shape[1]
    if (seq_lens.numel() != B or new_rows.numel() != B or blocks_in.numel() != B or blocks_out.numel() != B or
            (keep_blocks is not None and keep_blocks.numel() != B) or row_starts.numel() != B + 1 or slots.numel() != N or
            free_in.numel() < 1 or free_out.numel() != 2):
        raise ValueError("the lengths, the blocks, row_starts, positions, slots and the list's counts do not agree")
    dev = _device()
    _check(load().kv_plan_rows(
        _at(seq_lens, dev, _I32), _at(new_rows, dev, _I32), _at(block_tables, dev, _I32), _at(blocks_in, dev, _I32),
        _at(blocks_out, dev, _I32), _at(keep_blocks, dev, _I32), _at(free_list, dev, _I32), _at(free_in, dev, _I32),
        _at(free_out, dev, _I32), _at(row_starts, dev, _I32), _at(positions, dev, _I32), _at(slots, dev, _I64),
        _at(parents, dev, _I32), _at(tree_mask, dev, _I64), words, N, B, mbps, free_list.numel(), int(block_size),
        _raw_stream(dev) if stream is None else stream.cuda_stream), "kv_plan_rows")


def kv_append_slots(q, k_new, v_new, q_out, k_pool, v_pool, slots, positions=None, rope=None, q_weight=None, k_weight=None,
                    eps=1e-6, stream=None):
    """kv_append_paged_rows with each row's place given: row n is turned by positions[n] (int32 [N]) and its key
    and value go to slot slots[n] = block * bs + row of the pools (int64 [N]; below 0: the row is left out)."""
    N, Hkv, dk = k_new.shape
    nb, pool_heads, bs, dv = v_pool.shape
    H = 0
    if v_new.shape != (N, Hkv, dv) or k_pool.shape != (nb, Hkv, bs, dk) or pool_heads != Hkv:
        raise ValueError("k_new, v_new and the pools do not agree")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        H = q.shape[1]
        if q.shape != (N, H, dk) or q_out.shape != (N, H, dk):
            raise ValueError("q and q_out must both be [N, H, dk]")
        _writes_once(q_out)
    if slots.numel() != N or (positions is not None and positions.numel() != N):
        raise ValueError("slots and positions must be [N]")
    if (q_weight is not None and q_weight.shape != (dk,)) or (k_weight is not None and k_weight.shape != (dk,)):
        raise ValueError(f"a norm weight must be [{dk}]")
    dev = _device()
    dt = k_new.dtype
    for t in (k_new, v_new) if q is None else (q, k_new, v_new, q_out):
        if t.dtype is not dt:
            raise TypeError("tensors must share one dtype")
        if t.get_device() != dev:
            raise ValueError("tensors must live on the current CUDA device")
    if rope is not None and rope.table.get_device() != dev:
        raise ValueError("tensors must live on the current CUDA device")
    _check(load().kv_append_slots(
        _view(q, 3), _view(k_new, 3), _view(v_new, 3), _view(q_out, 3), _at(k_pool, dev, dt), _at(v_pool, dev, dt),
        _at(slots, dev, _I64), _at(positions, dev, _I32), N, nb, bs, H, Hkv, dk, dv, _at(q_weight, dev, dt),
        _at(k_weight, dev, dt), float(eps), _ref(rope), _number(dt), _raw_stream(dev) if stream is None else stream.cuda_stream),
           "kv_append_slots")
    return q_out


def attn_tree_paged_workspace_bytes(N, B, max_rows, max_len, H, Hkv, d_k, d_v, dtype=torch.bfloat16):
    return int(load().attn_tree_paged_workspace_bytes(N, B, max_rows, max_len, H, Hkv, d_k, d_v, _number(dtype)))


def tree_workspace(N, B, max_rows, H, Hkv, d_k, d_v, max_len, dtype=torch.bfloat16, device="cuda"):
    """A workspace tensor of the size attn_tree_paged needs (max_len: rows a table row can name); it does for smaller
    N, B, max_rows and max_len too."""
    return torch.empty(attn_tree_paged_workspace_bytes(N, B, max_rows, max_len, H, Hkv, d_k, d_v, dtype), dtype=torch.uint8,
                       device=device)


def attn_tree_paged(q, k_pool, v_pool, block_tables, position_offset, row_starts, tree_mask, out, attention_scale, max_rows,
                    workspace, stream=None, window=0, softcap=0.0, sinks=None, alibi_slopes=None):
    """Attention of drafted rows over the paged pool: rows row_starts[b] .. row_starts[b + 1] - 1 (int32 [B + 1], at most
    max_rows each) of q [N, H, dk] are sequence b's, lie in its cache behind position_offset[b] rows of history (int32
    [B] or None), and see that history and the drafted rows whose bits tree_mask int64 [N, words] sets (None: a chain,
    row i sees rows 0 .. i). pools [num_blocks, Hkv, bs, d]; block_tables int32 [B, mbps]; out [N, H, dv]; workspace from
    tree_workspace; window / softcap / sinks / alibi_slopes: the arms (`gqa_arms`). Rows of a sequence that kv_plan_rows
    could not serve get outputs that mean nothing."""
    N, H, dk = q.shape
    nb, Hkv, bs, dv = v_pool.shape
    B, mbps = block_tables.shape
    words = 0
    if tree_mask is not None:
        if tree_mask.dim() != 2 or tree_mask.shape[0] != N:
            raise ValueError("tree_mask must be [N, words]")
        words = tree_mask.shape[1]
    if (k_pool.shape != (nb, Hkv, bs, dk) or out.shape != (N, H, dv) or row_starts.numel() != B + 1 or
            (position_offset is not None and position_offset.numel() != B)):
        raise ValueError("q, the pools, the tables, the lengths, row_starts and out do not agree")
    dev = _device()
    arms = None
    if window or softcap or sinks is not None or alibi_slopes is not None:
        _here(sinks, alibi_slopes)
        if any(x is not None and x.numel() != H for x in (sinks, alibi_slopes)):
            raise ValueError("sinks and alibi_slopes must be float32 [H]")
        arms = _arms(window, softcap, sinks, alibi_slopes)
    dt, ws = q.dtype, 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("tensors must be contiguous and live on the current CUDA device")
        ws = workspace.numel() * workspace.element_size()
    _check(load().attn_tree_paged(
        _at(q, dev, dt), _at(k_pool, dev, dt), _at(v_pool, dev, dt), _at(block_tables, dev, _I32),
        _at(position_offset, dev, _I32), _at(row_starts, dev, _I32), _at(tree_mask, dev, _I64), _at(out, dev, dt), N, B,
        int(max_rows), words, mbps, nb, bs, H, Hkv, dk, dv, float(attention_scale), _number(dt), None if workspace is None else workspace.data_ptr(),
        ws, arms, _raw_stream(dev) if stream is None else stream.cuda_stream), "attn_tree_paged")
    return out


def kv_commit_rows(k_pools, v_pools, block_tables, seq_lens_in, row_starts, path, n_path, seq_lens_out, stream=None):
    """Moves row seq_lens_in[b] + path[b][j] to row seq_lens_in[b] + j, j < n_path[b], in every layer's pools
    (k_pools, v_pools: a tensor [num_blocks, Hkv, bs, d] each layer, or one of all layers [layers, num_blocks, ..],
    which is looked at once: 28 layers 14 us a call instead of 30; v_pools None: keys alone) and sets
    seq_lens_out[b] = seq_lens_in[b] + n_path[b] (may be the same tensor). path int32 [B, max_path], ascending
    indices among the row_starts[b + 1] - row_starts[b] drafted rows; n_path int32 [B] (0 for a sequence whose rows have
    no slots)."""
    layers = len(k_pools)
    B, mbps = block_tables.shape
    if not layers or (v_pools is not None and len(v_pools) != layers):
        raise ValueError("a pool of keys, and with values one of those, for each layer")

    def shape_of(pools):
        return pools.shape[1:] if isinstance(pools, torch.Tensor) else pools[0].shape

    k_shape, dt = shape_of(k_pools), k_pools.dtype if isinstance(k_pools, torch.Tensor) else k_pools[0].dtype
    nb, Hkv, bs, dk = k_shape
    v_shape = k_shape if v_pools is None else shape_of(v_pools)
    dv = 0 if v_pools is None else v_shape[3]
    if (v_shape[:3] != k_shape[:3] or len(v_shape) != 4 or path.dim() != 2 or path.shape[0] != B or row_starts.numel() != B + 1 or
            seq_lens_in.numel() != B or n_path.numel() != B or seq_lens_out.numel() != B):
        raise ValueError("the pools, the tables, the lengths and the paths do not agree")
    dev = block_tables.get_device()

    def addresses(pools, shape):
        if isinstance(pools, torch.Tensor):
            at, step = _at(pools, dev, dt), pools.stride(0) * pools.element_size()
            return struct.pack(f"{layers}Q", *range(at, at + layers * step, step))
        for x in pools:
            if x.shape != shape or x.dtype is not dt or x.get_device() != dev or not x.is_contiguous():
                raise ValueError("the layers' pools must be alike, contiguous and on one device")
        return struct.pack(f"{layers}Q", *[x.data_ptr() for x in pools])

    k_at = addresses(k_pools, k_shape)
    v_at = None if v_pools is None else addresses(v_pools, v_shape)
    if dev < 0 or dev != _device():
        raise ValueError("tensors must live on the current CUDA device")
    _check(load().kv_commit_rows(
        k_at, v_at, layers, _at(block_tables, dev, _I32),
        _at(seq_lens_in, dev, _I32), _at(row_starts, dev, _I32), _at(path, dev, _I32), _at(n_path, dev, _I32),
        _at(seq_lens_out, dev, _I32), B, path.shape[1], mbps, nb, bs, Hkv, dk, dv, _number(dt),
        _raw_stream(dev) if stream is None else stream.cuda_stream), "kv_commit_rows")


def attn_get_device_error(stream=None):
    """Synchronise the stream; return (and clear) the device error status code."""
    return int(load().attn_get_device_error(_stream(stream)))


def gqa_status_string(status):
    return load().gqa_status_string(int(status)).decode()


def gqa_debug_withhold_first_tile(enable):
    return int(load().gqa_debug_withhold_first_tile(int(bool(enable))))
