"""Sequence-mixer operators: recurrences over a chain of tokens.

Python binding of the entry points in ``include/selinv_seq.h``; like the rest
of the package it only marshals arguments.  The checks and the marshalling are
compiled (``csrc/seq_bind.cpp``), as a token's call is over in microseconds.

    y, state = short_conv(x, weight, bias, state=..., lengths=...)
    q, k = qk_norm_rotate(q, k, q_weight, k_weight, cos, sin, positions)
    y, state = selective_scan(x, dt, A, B, C, D, dt_bias, state=..., lengths=...)

Each has its reverse mode (``_vjp``: the cotangents of every output in, those of
every input out) and, where a state is carried, the form for one token per
sequence (``_step``), which updates a pool of states in place.

Token arrays are float32, float16 or bfloat16 and may be views (slices of a
fused projection) whose last dimension is contiguous; parameters are float32.
``lengths`` (int32, one per row) marks the tokens of a padded batch: outputs
and gradients past them are zero, and what stands there has no effect.
``slots`` (int32) names the state of each row in the pool; rows with a slot
outside the pool (-1: idle) get zeros and touch no state.

Like the package's other calls these record nothing for autograd: the gradients
are the ``_vjp`` calls (``examples/sequence_mixer.py`` wraps them as functions).
"""
from __future__ import annotations

import ctypes

import torch

_TYPES = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
MAX_W, MAX_HEAD, MAX_P, MAX_N = 8, 512, 256, 128
_bound = None  # the compiled binding, once it has the loaded library's addresses

_i64, _i32, _f32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p


def _struct(name, *fields):
    """A ctypes mirror of the C struct: (type, "names separated by blanks")."""
    return type(name, (ctypes.Structure,),
                {"_fields_": [(n, t) for t, names in fields for n in names.split()]})


ConvArgs = _struct(
    "ConvArgs", (_i64, "B T n_slots x_sb x_st yb_sb yb_st"), (_i32, "C W silu reserved"),
    (_vp, "x weight bias state lengths slots y state_out y_bar state_out_bar x_bar weight_bar "
          "bias_bar state_bar"))
QkrotArgs = _struct(
    "QkrotArgs", (_i64, "B T table_rows q_sb q_st q_sh k_sb k_st k_sh qb_sb qb_st qb_sh kb_sb "
                        "kb_st kb_sh pos_sb pos_st"),
    (_i32, "Hq Hk D R interleaved positions_64"), (_f32, "eps"), (_i32, "reserved"),
    (_vp, "q k q_weight k_weight cos_table sin_table positions q_out k_out q_bar k_bar q_grad "
          "k_grad q_weight_grad k_weight_grad"))
ScanArgs = _struct(
    "ScanArgs", (_i64, "B T n_slots x_sb x_st x_sh dt_sb dt_st b_sb b_st b_sg c_sb c_st c_sg "
                       "yb_sb yb_st yb_sh"),
    (_i32, "H P G N softplus reserved"),
    (_vp, "x dt Bm Cm A D dt_bias state lengths slots y state_out y_bar state_out_bar x_bar "
          "dt_bar B_bar C_bar A_bar D_bar dt_bias_bar state_bar"))


def declare(L):
    """Called when the library loads: ctypes signatures of the entry points."""
    release()
    sz = ctypes.c_size_t
    for sfx in _TYPES.values():
        for name, args in (("conv", ConvArgs), ("conv_step", ConvArgs), ("qkrot", QkrotArgs),
                           ("scan_step", ScanArgs)):
            f = getattr(L, "selinv_%s_%s" % (name, sfx))
            f.argtypes = [ctypes.POINTER(args), _vp]
            f.restype = ctypes.c_int
        for name, args in (("conv_vjp", ConvArgs), ("qkrot_vjp", QkrotArgs), ("scan", ScanArgs),
                           ("scan_vjp", ScanArgs)):
            f = getattr(L, "selinv_%s_%s" % (name, sfx))
            f.argtypes = [ctypes.POINTER(args), _vp, sz, _vp]
            f.restype = ctypes.c_int
    for name, args in (("conv_vjp", [_i64, _i64, _i32, _i32]), ("qkrot_vjp", [_i64, _i64, _i32]),
                       ("scan", [ctypes.c_int, _i64, _i64, _i32, _i32, _i32]),
                       ("scan_vjp", [ctypes.c_int, _i64, _i64, _i32, _i32, _i32, _i32]),
                       ("scan_vjp_bf16", [_i64, _i64, _i32, _i32, _i32, _i32])):
        f = getattr(L, "selinv_%s_workspace_bytes" % name)
        f.argtypes = args
        f.restype = sz


def release():
    """The library goes or is another one: the next call binds anew."""
    global _bound
    _bound = None


# the stream's handle without a Stream object around it, where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _binding():
    """The compiled binding.  The first call here loads it, and the library: the
    rest of the package does without it."""
    global _bound
    from . import _status, lib
    L = lib()
    try:
        from . import _seqbind
    except ImportError as e:
        raise ImportError("the binding of the sequence operators is not built for this Python and "
                          "torch (run sparse_spd_selected_amd.build())") from e
    _seqbind.bind(lambda name: ctypes.cast(getattr(L, name), _vp).value, _raw_stream, _status)
    _bound = _seqbind
    return _bound


# ------------------------------------------------------- short convolution
def short_conv(x, weight, bias=None, silu=True, state=None, lengths=None):
    """Short causal convolution of every channel.

    x [B, T, C]; weight [C, W] (the last tap meets the current token) and bias
    [C], float32; state [B, W-1, C] (x's type), the W - 1 tokens before the
    first, zeros if None; lengths [B].  Returns (y [B, T, C], state_out
    [B, W-1, C]): y = silu(bias + sum of taps), or without silu, and the last
    W - 1 tokens seen, to go on from.
    """
    return (_bound or _binding()).short_conv(x, weight, bias, silu, state, lengths)


def short_conv_step(x, state, weight, bias=None, silu=True, slots=None):
    """One token per row: x [B, C], state [n_slots, W-1, C] (x's type) updated
    in place, slots [B].  Returns y [B, C]."""
    return (_bound or _binding()).short_conv_step(x, state, weight, bias, silu, slots)


def short_conv_vjp(x, weight, bias, y_bar, state_out_bar=None, silu=True, state=None,
                   lengths=None):
    """Cotangents of (x, weight, bias, state) for a loss of short_conv's
    outputs: y_bar [B, T, C], state_out_bar [B, W-1, C] (None = 0).  The
    forward is recomputed.  Returns (x_bar, weight_bar, bias_bar, state_bar);
    bias_bar and state_bar are None where there is no bias or state."""
    return (_bound or _binding()).short_conv_vjp(x, weight, bias, y_bar, state_out_bar, silu,
                                                 state, lengths)


# ------------------------------------------------- head norm and rotation
def qk_norm_rotate(q, k, q_weight, k_weight, cos=None, sin=None, positions=None, eps=1e-6,
                   interleaved=False):
    """Root-mean-square norm of every query and key head and its rotation by
    position, in one pass.

    q [B, T, Hq, D], k [B, T, Hk, D] (or None), q_weight, k_weight [D]
    float32; cos, sin [rows, R/2] float32, the table of the rotation's angles,
    and positions [B, T] (or broadcastable to it; int32 or int64) into it.  The
    first R elements of a head turn, as halves (i, i + R/2) or, interleaved, as
    neighbours (2i, 2i + 1); without cos nothing does.  A token whose position
    is outside the table comes out as NaN.  Returns (q_out, k_out), contiguous.
    """
    return (_bound or _binding()).qk_norm_rotate(q, k, q_weight, k_weight, cos, sin, positions, eps,
                                                 interleaved)


def qk_norm_rotate_vjp(q, k, q_weight, k_weight, cos, sin, positions, q_out_bar, k_out_bar,
                       eps=1e-6, interleaved=False):
    """Cotangents of (q, k, q_weight, k_weight) for a loss of
    qk_norm_rotate's outputs, given theirs."""
    return (_bound or _binding()).qk_norm_rotate_vjp(q, k, q_weight, k_weight, cos, sin, positions,
                                                     q_out_bar, k_out_bar, eps, interleaved)


# --------------------------------------------------------- selective scan
def selective_scan(x, dt, A, Bm, Cm, D=None, dt_bias=None, softplus=True, state=None,
                   lengths=None):
    """Selective state space scan: for every head, with a P x N state S,

        d_t = softplus(dt_t + dt_bias)        (or dt_t + dt_bias)
        S_t = exp(d_t A) S_{t-1} + d_t x_t B_t^T
        y_t = S_t C_t + D x_t

    x [B, T, H, P], dt [B, T, H], Bm, Cm [B, T, G, N] (H a multiple of G); A,
    D, dt_bias [H] float32; state [B, H, P, N] float32, zeros if None; lengths
    [B].  Returns (y [B, T, H, P], state_out [B, H, P, N] float32)."""
    return (_bound or _binding()).selective_scan(x, dt, A, Bm, Cm, D, dt_bias, softplus, state,
                                                 lengths)


def selective_scan_step(x, dt, A, Bm, Cm, state, D=None, dt_bias=None, softplus=True, slots=None):
    """One token per row: x [B, H, P], dt [B, H], Bm, Cm [B, G, N], state
    [n_slots, H, P, N] float32 updated in place, slots [B].  Returns y
    [B, H, P]."""
    return (_bound or _binding()).selective_scan_step(x, dt, A, Bm, Cm, state, D, dt_bias, softplus,
                                                      slots)


def selective_scan_vjp(x, dt, A, Bm, Cm, y_bar, state_out_bar=None, D=None, dt_bias=None,
                       softplus=True, state=None, lengths=None):
    """Cotangents of (x, dt, A, Bm, Cm, D, dt_bias, state) for a loss of
    selective_scan's outputs: y_bar [B, T, H, P], state_out_bar [B, H, P, N]
    float32 (None = 0).  The forward is recomputed; the workspace holds two
    float32 states per head and chunk of 32 tokens (bfloat16: 64).  D's, dt_bias's and state's
    are None where those are."""
    return (_bound or _binding()).selective_scan_vjp(x, dt, A, Bm, Cm, y_bar, state_out_bar, D,
                                                     dt_bias, softplus, state, lengths)
