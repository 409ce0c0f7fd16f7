"""Thin ctypes binding of libflashcart (C ABI in include/flashcart.h).

Argument marshalling only: tensors are checked for device, dtype and shape,
their device pointers and the current CUDA stream are handed to the C entry
points, and a non-zero status becomes a FlashCartError.  Every step of the
computation runs in the library's CUDA kernels; there is no fallback.  If the
library has not been built this module raises on import.

Conventions (layouts, path order, component order) are those of the header.
"""
import ctypes as ct
import functools
import inspect
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libflashcart.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "libflashcart.so is not built (expected at %s); run "
        "`python -m cartesian_tensor_products_b200.build`" % LIB_PATH)

_lib = ct.CDLL(LIB_PATH)

FC_OK = 0


class FlashCartError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (status %d)" % (
            where, _lib.fc_status_string(status).decode(), status))


class ConvDesc(ct.Structure):
    _fields_ = [("lmax_in", ct.c_int), ("lmax_edge", ct.c_int),
                ("lmax_out", ct.c_int), ("channels", ct.c_int),
                ("sum_paths", ct.c_int), ("envelope", ct.c_int),
                ("r_cut", ct.c_float), ("edge_scale", ct.c_float)]


class LadderDesc(ct.Structure):
    _fields_ = [("lmax", ct.c_int), ("channels", ct.c_int), ("order", ct.c_int)]


class HeadDesc(ct.Structure):
    __hash__ = object.__hash__     # by identity: cached scratch sizes are looked up by it
    _fields_ = [("dtype", ct.c_int), ("heads_q", ct.c_int), ("heads_k", ct.c_int),
                ("head_dim", ct.c_int), ("pairs", ct.c_int), ("eps", ct.c_float)]


class AttnDesc(ct.Structure):
    __hash__ = object.__hash__
    _fields_ = [("dtype", ct.c_int), ("heads", ct.c_int), ("kv_heads", ct.c_int),
                ("head_dim", ct.c_int), ("scale", ct.c_float), ("cap", ct.c_float)]


_vp = ct.c_void_p
_SIGS = {
    "fc_status_string": (ct.c_char_p, [ct.c_int]),
    "fc_version": (ct.c_int, []),
    "fc_conv_num_paths": (ct.c_int, [ct.POINTER(ConvDesc)]),
    "fc_conv_out_row": (ct.c_int, [ct.POINTER(ConvDesc)]),
    "fc_conv_path": (ct.c_int, [ct.POINTER(ConvDesc), ct.c_int, ct.POINTER(ct.c_int),
                                ct.POINTER(ct.c_int), ct.POINTER(ct.c_int)]),
    "fc_build_rowptr": (ct.c_int, [ct.c_int, ct.c_int, _vp, _vp, _vp, _vp, _vp]),
    "fc_build_rowptr_rect": (ct.c_int, [ct.c_int, ct.c_int, ct.c_int, _vp, _vp, _vp, _vp, _vp]),
    "fc_edge_conv": (ct.c_int, [ct.POINTER(ConvDesc), ct.c_int, ct.c_int,
                                _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fc_edge_conv_rect": (ct.c_int, [ct.POINTER(ConvDesc), ct.c_int, ct.c_int, ct.c_int,
                                     _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fc_edge_conv_vjp": (ct.c_int, [ct.POINTER(ConvDesc), ct.c_int, ct.c_int,
                                    _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fc_edge_conv_vjp_rect": (ct.c_int, [ct.POINTER(ConvDesc), ct.c_int, ct.c_int, ct.c_int,
                                         _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fc_conv_odd_num_paths": (ct.c_int, [ct.POINTER(ConvDesc)]),
    "fc_conv_odd_out_row": (ct.c_int, [ct.POINTER(ConvDesc)]),
    "fc_conv_odd_path": (ct.c_int, [ct.POINTER(ConvDesc), ct.c_int, ct.POINTER(ct.c_int),
                                    ct.POINTER(ct.c_int), ct.POINTER(ct.c_int)]),
    "fc_edge_conv_odd": (ct.c_int, [ct.POINTER(ConvDesc), ct.c_int, ct.c_int,
                                    _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fc_edge_conv_odd_vjp": (ct.c_int, [ct.POINTER(ConvDesc), ct.c_int, ct.c_int,
                                        _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fc_scalar_readout": (ct.c_int, [ct.c_int, ct.c_int, ct.c_int, _vp, _vp, _vp, _vp]),
    "fc_edge_forces": (ct.c_int, [ct.c_int, ct.c_int, _vp, _vp, _vp, _vp]),
    "fc_ladder_num_paths": (ct.c_int, [ct.POINTER(LadderDesc)]),
    "fc_product_ladder_workspace_size": (ct.c_size_t, [ct.POINTER(LadderDesc), ct.c_int]),
    "fc_product_ladder": (ct.c_int, [ct.POINTER(LadderDesc), ct.c_int, _vp, _vp, _vp, _vp,
                                     _vp, _vp, ct.c_size_t, _vp]),
    "fc_product_ladder_vjp_workspace_size": (ct.c_size_t, [ct.POINTER(LadderDesc), ct.c_int]),
    "fc_product_ladder_vjp": (ct.c_int, [ct.POINTER(LadderDesc), ct.c_int, _vp, _vp, _vp, _vp,
                                         _vp, _vp, _vp, _vp, _vp, ct.c_size_t, _vp]),
    "fc_device_error": (ct.c_int, [ct.POINTER(ct.c_int), _vp]),
    "fc_set_wait_timeout": (ct.c_int, [ct.c_uint64]),
    "fc_edge_conv_workspace_size": (ct.c_size_t, [ct.POINTER(ConvDesc), ct.c_int, ct.c_int]),
    "fc_edge_conv_vjp_vjp": (ct.c_int, [ct.POINTER(ConvDesc), ct.c_int, ct.c_int] + [_vp] * 14),
    "fc_full_ladder_workspace_size": (ct.c_size_t, [ct.POINTER(LadderDesc), ct.c_int]),
    "fc_full_ladder": (ct.c_int, [ct.POINTER(LadderDesc), ct.c_int, _vp, _vp, _vp, _vp, _vp, _vp,
                                  ct.c_size_t, _vp]),
    "fc_full_ladder_vjp_workspace_size": (ct.c_size_t, [ct.POINTER(LadderDesc), ct.c_int]),
    "fc_full_ladder_vjp": (ct.c_int, [ct.POINTER(LadderDesc), ct.c_int] + [_vp] * 9
                           + [ct.c_size_t, _vp]),
    "fc_species_embed": (ct.c_int, [ct.c_int] * 5 + [ct.c_float] + [_vp] * 4),
    "fc_species_embed_vjp_workspace_size": (ct.c_size_t, [ct.c_int] * 3),
    "fc_species_embed_vjp": (ct.c_int, [ct.c_int] * 5 + [ct.c_float] + [_vp] * 4
                             + [ct.c_size_t, _vp]),
    "fc_head_norm_rotate": (ct.c_int, [ct.POINTER(HeadDesc), ct.c_int, _vp, ct.c_int64]
                            + [_vp] * 5 + [ct.c_int64, _vp]),
    "fc_head_norm_rotate_vjp_workspace_size": (ct.c_size_t, [ct.POINTER(HeadDesc), ct.c_int]),
    "fc_head_norm_rotate_vjp": (ct.c_int, [ct.POINTER(HeadDesc), ct.c_int, _vp, ct.c_int64, _vp,
                                           ct.c_int64] + [_vp] * 5 + [ct.c_int64] + [_vp] * 4
                                + [ct.c_size_t, _vp]),
    "fc_node_attention_workspace_size": (ct.c_size_t, [ct.POINTER(AttnDesc)] + [ct.c_int] * 3),
    "fc_node_attention_on_tcgen05": (ct.c_int, [ct.POINTER(AttnDesc)] + [ct.c_int] * 4),
    "fc_node_attention": (ct.c_int, [ct.POINTER(AttnDesc)] + [ct.c_int] * 3 + [_vp] * 2
                          + [_vp, ct.c_int64] * 3 + [_vp] * 4 + [_vp, ct.c_int64] + [_vp] * 3
                          + [ct.c_size_t, _vp]),
    "fc_node_attention_vjp_workspace_size": (ct.c_size_t, [ct.POINTER(AttnDesc)] + [ct.c_int] * 3),
    "fc_node_attention_vjp": (ct.c_int, [ct.POINTER(AttnDesc)] + [ct.c_int] * 3 + [_vp] * 2
                              + [_vp, ct.c_int64] * 3 + [_vp] * 6 + [_vp, ct.c_int64] + [_vp] * 7
                              + [ct.c_size_t, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def lib():
    return _lib


def _check(status, where):
    if status != FC_OK:
        raise FlashCartError(status, where)


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return _vp(stream.cuda_stream)


def _ptr(t):
    return _vp(t.data_ptr()) if t is not None else None


def _dev(t, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def conv_desc(lmax, channels, sum_paths=False, envelope=None):
    """envelope: None, or (r_cut, edge_scale) for the cosine radial envelope."""
    if envelope is None:
        return ConvDesc(lmax, lmax, lmax, channels, int(bool(sum_paths)), 0, 0.0, 0.0)
    r_cut, scale = envelope
    return ConvDesc(lmax, lmax, lmax, channels, int(bool(sum_paths)), 1, float(r_cut),
                    float(scale))


def num_paths(lmax, channels=4, sum_paths=False):
    d = conv_desc(lmax, channels, sum_paths)
    n = _lib.fc_conv_num_paths(ct.byref(d))
    if n < 0:
        raise FlashCartError(4, "fc_conv_num_paths")
    return n


def out_row(lmax, channels=4, sum_paths=False):
    d = conv_desc(lmax, channels, sum_paths)
    n = _lib.fc_conv_out_row(ct.byref(d))
    if n < 0:
        raise FlashCartError(4, "fc_conv_out_row")
    return n


def paths(lmax):
    d = conv_desc(lmax, 4)
    out = []
    for p in range(num_paths(lmax)):
        a, b, c = ct.c_int(), ct.c_int(), ct.c_int()
        _check(_lib.fc_conv_path(ct.byref(d), p, ct.byref(a), ct.byref(b), ct.byref(c)),
               "fc_conv_path")
        out.append((a.value, b.value, c.value))
    return out


def odd_num_paths(lmax, channels=4, sum_paths=False):
    """Number of odd-J (Levi-Civita) paths at this rank."""
    d = conv_desc(lmax, channels, sum_paths)
    n = _lib.fc_conv_odd_num_paths(ct.byref(d))
    if n < 0:
        raise FlashCartError(4, "fc_conv_odd_num_paths")
    return n


def odd_out_row(lmax, channels=4, sum_paths=False):
    d = conv_desc(lmax, channels, sum_paths)
    n = _lib.fc_conv_odd_out_row(ct.byref(d))
    if n < 0:
        raise FlashCartError(4, "fc_conv_odd_out_row")
    return n


def odd_paths(lmax):
    d = conv_desc(lmax, 4)
    out = []
    for p in range(odd_num_paths(lmax)):
        a, b, c = ct.c_int(), ct.c_int(), ct.c_int()
        _check(_lib.fc_conv_odd_path(ct.byref(d), p, ct.byref(a), ct.byref(b), ct.byref(c)),
               "fc_conv_odd_path")
        out.append((a.value, b.value, c.value))
    return out


def build_rowptr(edge_index, edge_vec, n_nodes, stream=None, n_send=None):
    """Receiver row pointer [n_nodes+1] of a receiver-sorted edge list; raises
    FlashCartError(FC_ERR_CSR / FC_ERR_DEGENERATE_EDGE) on a bad graph.
    n_send: sender count when it differs from the receiver count (a
    receiver range of a larger graph)."""
    _dev(edge_index, torch.int32, "edge_index")
    E = edge_index.shape[1]
    if edge_vec is not None:
        _dev(edge_vec, torch.float32, "edge_vec")
        assert edge_vec.shape == (E, 3)
    dev = edge_index.device
    rowptr = torch.empty(n_nodes + 1, dtype=torch.int32, device=dev)
    flag = torch.empty(1, dtype=torch.int32, device=dev)
    _check(_lib.fc_build_rowptr_rect(n_nodes, n_nodes if n_send is None else n_send, E,
                                     _ptr(edge_index), _ptr(edge_vec), _ptr(rowptr), _ptr(flag),
                                     _stream(stream)), "fc_build_rowptr")
    return rowptr


def edge_conv(lmax, rowptr, edge_index, edge_vec, x, w, sum_paths=False,
              out=None, stream=None, envelope=None, odd=False):
    """z of Sec. 4 Eq. (1): [N][out_row * C].  odd=True: over the odd-J
    (Levi-Civita) paths (fc_edge_conv_odd; senders = receivers)."""
    _dev(rowptr, torch.int32, "rowptr")
    _dev(edge_index, torch.int32, "edge_index")
    _dev(edge_vec, torch.float32, "edge_vec")
    _dev(x, torch.float32, "x")
    _dev(w, torch.float32, "w")
    N = rowptr.shape[0] - 1
    E = edge_index.shape[1]
    C = x.shape[1] // ((lmax + 1) ** 2)
    d = conv_desc(lmax, C, sum_paths, envelope)
    zr = odd_out_row(lmax, C, sum_paths) if odd else out_row(lmax, C, sum_paths)
    NS = x.shape[0]     # senders: N, or all nodes of the graph for a receiver range
    if x.dim() != 2 or x.shape[1] != (lmax + 1) ** 2 * C:
        raise ValueError("x shape %s" % (tuple(x.shape),))
    if w.numel() != E * (odd_num_paths(lmax) if odd else num_paths(lmax)) * C:
        raise ValueError("w shape %s" % (tuple(w.shape),))
    if out is None:
        out = torch.empty((N, zr * C), dtype=torch.float32, device=x.device)
    else:
        _dev(out, torch.float32, "out")
        assert out.shape == (N, zr * C)
    if odd:
        if NS != N:
            raise ValueError("the odd-J convolution takes senders = receivers")
        _check(_lib.fc_edge_conv_odd(ct.byref(d), N, E, _ptr(rowptr), _ptr(edge_index),
                                     _ptr(edge_vec), _ptr(x), _ptr(w), _ptr(out),
                                     _stream(stream)), "fc_edge_conv_odd")
        return out
    _check(_lib.fc_edge_conv_rect(ct.byref(d), N, NS, E, _ptr(rowptr), _ptr(edge_index),
                                  _ptr(edge_vec), _ptr(x), _ptr(w), _ptr(out),
                                  _stream(stream)), "fc_edge_conv")
    return out


def edge_conv_vjp(lmax, rowptr, edge_index, edge_vec, x, w, g, sum_paths=False,
                  want=("x", "w", "r"), out=None, stream=None, envelope=None, odd=False):
    """(x_bar, w_bar, r_bar) of App. C Eq. (C1); entries not in `want` are None.
    odd=True: the VJP of the odd-J path convolution."""
    _dev(rowptr, torch.int32, "rowptr")
    _dev(edge_index, torch.int32, "edge_index")
    _dev(edge_vec, torch.float32, "edge_vec")
    _dev(x, torch.float32, "x")
    _dev(w, torch.float32, "w")
    _dev(g, torch.float32, "g")
    N = rowptr.shape[0] - 1
    E = edge_index.shape[1]
    C = x.shape[1] // ((lmax + 1) ** 2)
    d = conv_desc(lmax, C, sum_paths, envelope)
    P = odd_num_paths(lmax) if odd else num_paths(lmax)
    zr = odd_out_row(lmax, C, sum_paths) if odd else out_row(lmax, C, sum_paths)
    if g.shape != (N, zr * C):
        raise ValueError("g shape %s" % (tuple(g.shape),))
    if out is None:
        out = {}
    xb = out.get("x") if "x" in want else None
    wb = out.get("w") if "w" in want else None
    rb = out.get("r") if "r" in want else None
    if "x" in want and xb is None:
        xb = torch.empty_like(x)
    if "w" in want and wb is None:
        wb = torch.empty((E, P, C), dtype=torch.float32, device=x.device)
    if "r" in want and rb is None:
        rb = torch.empty((E, 3), dtype=torch.float32, device=x.device)
    if odd:
        _check(_lib.fc_edge_conv_odd_vjp(ct.byref(d), N, E, _ptr(rowptr), _ptr(edge_index),
                                         _ptr(edge_vec), _ptr(x), _ptr(w), _ptr(g), _ptr(xb),
                                         _ptr(wb), _ptr(rb), _stream(stream)), "fc_edge_conv_odd_vjp")
        return xb, wb, rb
    _check(_lib.fc_edge_conv_vjp_rect(ct.byref(d), N, x.shape[0], E, _ptr(rowptr), _ptr(edge_index),
                                      _ptr(edge_vec), _ptr(x), _ptr(w), _ptr(g), _ptr(xb),
                                      _ptr(wb), _ptr(rb), _stream(stream)), "fc_edge_conv_vjp")
    return xb, wb, rb


def edge_conv_vjp_vjp(lmax, rowptr, edge_index, edge_vec, x, w, g, v_x=None, v_w=None,
                      v_r=None, sum_paths=False, want=("g", "x", "w", "r"), stream=None):
    """(g_hat, x_hat, w_hat, r_hat) of App. C Eq. C2 (Algorithm 3): the
    gradients of <v_x, x_bar> + <v_w, w_bar> + <v_r, r_bar> with respect to
    g, x, w and the edge vectors; None cotangents are zero, outputs not in
    `want` are None."""
    for t, n in ((x, "x"), (g, "g")):
        _dev(t, torch.float32, n)
    _dev(rowptr, torch.int32, "rowptr")
    _dev(edge_index, torch.int32, "edge_index")
    for t, n in ((v_x, "v_x"), (v_w, "v_w"), (v_r, "v_r")):
        if t is not None:
            _dev(t, torch.float32, n)
    N = rowptr.shape[0] - 1
    E = edge_index.shape[1]
    C = x.shape[1] // ((lmax + 1) ** 2)
    d = conv_desc(lmax, C, sum_paths)
    P = num_paths(lmax)
    if g.shape != (N, out_row(lmax, C, sum_paths) * C):
        raise ValueError("g shape %s" % (tuple(g.shape),))
    gh = torch.empty_like(g) if "g" in want else None
    xh = torch.empty_like(x) if "x" in want else None
    wh = torch.empty((E, P, C), dtype=torch.float32, device=x.device) if "w" in want else None
    rh = torch.empty((E, 3), dtype=torch.float32, device=x.device) if "r" in want else None
    _check(_lib.fc_edge_conv_vjp_vjp(ct.byref(d), N, E, _ptr(rowptr), _ptr(edge_index),
                                     _ptr(edge_vec), _ptr(x), _ptr(w), _ptr(g), _ptr(v_x),
                                     _ptr(v_w), _ptr(v_r), _ptr(gh), _ptr(xh), _ptr(wh),
                                     _ptr(rh), _stream(stream)), "fc_edge_conv_vjp_vjp")
    return gh, xh, wh, rh


def _workspace(nbytes, device):
    if nbytes == 0:
        return None
    return torch.empty((nbytes + 15) // 16 * 4, dtype=torch.float32, device=device)


def _scratch(workspace, need, device):
    """(buffer, its size in bytes): a new buffer of `need` bytes, or the
    caller's tensor with its actual size, which the library checks."""
    if workspace is None:
        return _workspace(need, device), need
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace, workspace.numel() * workspace.element_size()


def ladder_workspace_bytes(lmax, channels, order, n_nodes, vjp=False):
    """Scratch bytes fc_product_ladder (or, with vjp=True, its VJP) needs."""
    d = LadderDesc(lmax, channels, order)
    f = _lib.fc_product_ladder_vjp_workspace_size if vjp else _lib.fc_product_ladder_workspace_size
    return f(ct.byref(d), n_nodes)


def product_ladder(lmax, order, A1, path_w, mix_w, workspace=None, stream=None):
    """(states [order-1][N][...], z) of Sec. 5 Eq. (2), path-reduced products
    followed by a per-rank channel mix."""
    _dev(A1, torch.float32, "A1")
    N = A1.shape[0]
    NY = (lmax + 1) ** 2
    C = A1.shape[1] // NY
    d = LadderDesc(lmax, C, order)
    S = order - 1
    states = torch.empty((max(S, 0), N, NY * C), dtype=torch.float32, device=A1.device)
    z = torch.empty_like(A1)
    ws_bytes = _lib.fc_product_ladder_workspace_size(ct.byref(d), N)
    workspace, ws_bytes = _scratch(workspace, ws_bytes, A1.device)
    if S > 0:
        _dev(path_w, torch.float32, "path_w")
        _dev(mix_w, torch.float32, "mix_w")
    _check(_lib.fc_product_ladder(ct.byref(d), N, _ptr(A1), _ptr(path_w) if S > 0 else None,
                                  _ptr(mix_w) if S > 0 else None, _ptr(states) if S > 0 else None,
                                  _ptr(z), _ptr(workspace), ws_bytes if workspace is not None else 0,
                                  _stream(stream)), "fc_product_ladder")
    return states, z


def product_ladder_vjp(lmax, order, A1, path_w, mix_w, states, gz, workspace=None,
                       stream=None):
    """(A1_bar, path_w_bar, mix_w_bar) of fc_product_ladder."""
    _dev(A1, torch.float32, "A1")
    _dev(gz, torch.float32, "gz")
    N = A1.shape[0]
    NY = (lmax + 1) ** 2
    C = A1.shape[1] // NY
    d = LadderDesc(lmax, C, order)
    S = order - 1
    A1b = torch.empty_like(A1)
    pwb = torch.empty((max(S, 0),) + tuple(path_w.shape[1:]), dtype=torch.float32, device=A1.device)
    mwb = torch.empty((max(S, 0),) + tuple(mix_w.shape[1:]), dtype=torch.float32, device=A1.device)
    ws_bytes = _lib.fc_product_ladder_vjp_workspace_size(ct.byref(d), N)
    workspace, ws_bytes = _scratch(workspace, ws_bytes, A1.device)
    _check(_lib.fc_product_ladder_vjp(
        ct.byref(d), N, _ptr(A1), _ptr(path_w) if S > 0 else None,
        _ptr(mix_w) if S > 0 else None, _ptr(states) if S > 0 else None, _ptr(gz),
        _ptr(A1b), _ptr(pwb) if S > 0 else None, _ptr(mwb) if S > 0 else None,
        _ptr(workspace), ws_bytes if workspace is not None else 0, _stream(stream)),
        "fc_product_ladder_vjp")
    return A1b, pwb, mwb


def full_ladder(lmax, order, A, W1, Wq, workspace=None, stream=None):
    """(states [order][N][...] = phi_1..phi_order, z) of the full ladder
    (Sec. 5 Eq. 2): path-separated products, per-rank path+channel maps."""
    _dev(A, torch.float32, "A")
    _dev(W1, torch.float32, "W1")
    N = A.shape[0]
    NY = (lmax + 1) ** 2
    C = A.shape[1] // NY
    d = LadderDesc(lmax, C, order)
    states = torch.empty((order, N, NY * C), dtype=torch.float32, device=A.device)
    z = torch.empty_like(A)
    if order > 1:
        _dev(Wq, torch.float32, "Wq")
    ws_bytes = _lib.fc_full_ladder_workspace_size(ct.byref(d), N)
    workspace, ws_bytes = _scratch(workspace, ws_bytes, A.device)
    _check(_lib.fc_full_ladder(ct.byref(d), N, _ptr(A), _ptr(W1), _ptr(Wq) if order > 1 else None,
                               _ptr(states), _ptr(z), _ptr(workspace),
                               ws_bytes if workspace is not None else 0, _stream(stream)),
           "fc_full_ladder")
    return states, z


def full_ladder_vjp(lmax, order, A, W1, Wq, states, gz, workspace=None, stream=None):
    """(A_bar, W1_bar, Wq_bar): gradients of <gz, z> for fc_full_ladder,
    given the states phi_1..phi_order it returned."""
    for t, n in ((A, "A"), (W1, "W1"), (states, "states"), (gz, "gz")):
        _dev(t, torch.float32, n)
    N = A.shape[0]
    NY = (lmax + 1) ** 2
    C = A.shape[1] // NY
    d = LadderDesc(lmax, C, order)
    Ab = torch.empty_like(A)
    W1b = torch.empty_like(W1)
    if order > 1:
        _dev(Wq, torch.float32, "Wq")
        Wqb = torch.empty_like(Wq)
    else:
        Wqb = None
    ws_bytes = _lib.fc_full_ladder_vjp_workspace_size(ct.byref(d), N)
    workspace, ws_bytes = _scratch(workspace, ws_bytes, A.device)
    _check(_lib.fc_full_ladder_vjp(ct.byref(d), N, _ptr(A), _ptr(W1), _ptr(Wq) if order > 1 else None,
                                   _ptr(states), _ptr(gz), _ptr(Ab), _ptr(W1b), _ptr(Wqb),
                                   _ptr(workspace), ws_bytes if workspace is not None else 0,
                                   _stream(stream)), "fc_full_ladder_vjp")
    return Ab, W1b, Wqb


def device_error(stream=None):
    """Sticky error word of the kernels with bounded barrier waits (0 = none
    gave up since the last call); synchronises the stream and clears it."""
    flag = ct.c_int(0)
    _check(_lib.fc_device_error(ct.byref(flag), _stream(stream)), "fc_device_error")
    return flag.value


def set_wait_timeout(ns=0):
    """Bound (ns) of the tensor-core kernels' barrier waits on the current
    device; 0 restores the default."""
    _check(_lib.fc_set_wait_timeout(int(ns)), "fc_set_wait_timeout")


def scalar_readout(lmax, z, want_grad=True, stream=None):
    """(energy [1], gz) with energy = sum of the rank-0 block of z and
    gz = d energy / d z."""
    _dev(z, torch.float32, "z")
    N = z.shape[0]
    C = z.shape[1] // ((lmax + 1) ** 2)
    energy = torch.empty(1, dtype=torch.float32, device=z.device)
    gz = torch.empty_like(z) if want_grad else None
    _check(_lib.fc_scalar_readout(N, lmax, C, _ptr(z), _ptr(energy), _ptr(gz),
                                  _stream(stream)), "fc_scalar_readout")
    return energy, gz


def edge_forces(edge_index, r_bar, n_nodes, stream=None):
    """forces [N][3] = -dE/dpos from per-edge gradients r_bar."""
    _dev(edge_index, torch.int32, "edge_index")
    _dev(r_bar, torch.float32, "r_bar")
    F = torch.empty((n_nodes, 3), dtype=torch.float32, device=r_bar.device)
    _check(_lib.fc_edge_forces(n_nodes, edge_index.shape[1], _ptr(edge_index), _ptr(r_bar),
                               _ptr(F), _stream(stream)), "fc_edge_forces")
    return F


def interaction_block(lmax, order, rowptr, edge_index, edge_vec, x, omega, path_w, mix_w,
                      r_cut, edge_scale, stream=None):
    """Energy and forces of one interaction block, each step a library call:
    edge convolution with paths summed per output rank and the cosine
    envelope (App. E Eq. E1 with the 1/sqrt(mean neighbours) factor in
    edge_scale), the product ladder (Sec. 5 Eq. 2), E = sum of its rank-0
    outputs, then the ladder VJP, the convolution VJP (r_bar only) and the
    force scatter.  Returns (energy [1], forces [N][3], z)."""
    env = (r_cut, edge_scale)
    N = rowptr.shape[0] - 1
    A1 = edge_conv(lmax, rowptr, edge_index, edge_vec, x, omega, sum_paths=True,
                   envelope=env, stream=stream)
    states, z = product_ladder(lmax, order, A1, path_w, mix_w, stream=stream)
    energy, gz = scalar_readout(lmax, z, stream=stream)
    A1b, _, _ = product_ladder_vjp(lmax, order, A1, path_w, mix_w, states, gz, stream=stream)
    _, _, rb = edge_conv_vjp(lmax, rowptr, edge_index, edge_vec, x, omega, A1b, sum_paths=True,
                             want=("r",), envelope=env, stream=stream)
    F = edge_forces(edge_index, rb, N, stream=stream)
    return energy, F, z


# ----------------------------------------------------------------------------
# operators on node rows (include/flashcart_nodes.h)
#
# These calls are often a few microseconds of GPU work, so that the checks
# below are written to cost little: plain integers for pointers and stream,
# descriptors and scratch sizes looked up by their values.

_F32, _U8, _I32 = torch.float32, torch.uint8, torch.int32
_ROW_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _node_op(f):
    """Runs a node operator on its first tensor's device and on `stream` (None:
    that device's current stream), which f gets as the raw handle.  Outputs and
    scratch are allocated on the stream that uses them."""
    name = next(iter(inspect.signature(f).parameters))

    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise TypeError("%s takes CUDA tensors" % f.__name__)
        index = first.get_device()
        if stream is None and index == torch._C._cuda_getDevice():
            return f(*args, stream=torch._C._cuda_getCurrentRawStream(index), **kw)
        if stream is not None and stream.device.index != index:
            raise ValueError("stream is on %s, the tensors are on %s" % (stream.device, first.device))
        with torch.cuda.device(index), torch.cuda.stream(stream):
            return f(*args, stream=torch._C._cuda_getCurrentRawStream(index), **kw)
    return call


def _on(t, dtype, name, index, shape):
    """Address of a contiguous tensor on device `index`; None passes as NULL.  A
    tensor without elements has address 0, which would read as None: it passes
    as an aligned address that nothing follows."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, index))
    if t.shape != shape:
        raise ValueError("%s shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr() or 16


def _counts(*sizes):
    """Sizes as the library takes them: ctypes would drop the bits from 32 on."""
    for n in sizes:
        if not 0 <= n < 1 << 31:
            raise ValueError("size %d is outside 0 .. 2^31 - 1" % n)


def _row_dtype(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    d = _ROW_DTYPES.get(t.dtype)
    if d is None:
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, t.dtype))
    return d


def _rows(t, name, dtype, index, shape):
    """(address, row step) of [N][heads][head_dim] rows: the heads of a row are
    packed, rows may be a column block of a wider array."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, index))
    if t.shape != shape:
        raise ValueError("%s shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    n, h, d = shape
    sn, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError("%s: the heads of a row must be packed" % name)
    return t.data_ptr(), sn if n > 1 else h * d


def _rows3(t, name):
    if t.dim() != 3:
        raise ValueError("%s shape %s, expected [nodes][heads][head_dim]" % (name, tuple(t.shape)))
    return t.shape


@functools.lru_cache(maxsize=256)
def _scratch_size(index, query, desc, *sizes):
    f = getattr(_lib, query)
    return f(desc, *sizes) if desc is not None else f(*sizes)


def _bytes(workspace, need, index):
    """(tensor, address, size) of scratch: a new buffer of `need` bytes, or the
    caller's with its real size."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=_U8, device=index)
        return workspace, workspace.data_ptr(), need
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if workspace.get_device() != index:
        raise ValueError("workspace is on %s, expected cuda:%d" % (workspace.device, index))
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


@_node_op
def species_embed(species, table, lmax=0, scale=1.0, out=None, stream=None):
    """Node features [N][(lmax+1)^2 C] of the species (int32 [N]): scale times
    the table's row [n_species][C] in the rank-0 block, zero elsewhere.  A
    species outside the table (padding: -1) gets a zero row."""
    index, dtype = species.get_device(), _row_dtype(table, "table")
    if species.dim() != 1 or table.dim() != 2:
        raise ValueError("species [N] and table [n_species][C] expected")
    (N,), (V, C) = species.shape, table.shape
    _counts(N, V, C, lmax)
    shape = (N, (lmax + 1) ** 2 * C)
    if out is None:
        out = table.new_empty(shape)
    _check(_lib.fc_species_embed(dtype, N, V, lmax, C, scale, _on(species, _I32, "species", index, (N,)),
                                 _on(table, table.dtype, "table", index, (V, C)),
                                 _on(out, table.dtype, "out", index, shape), stream), "fc_species_embed")
    return out


@_node_op
def species_embed_vjp(species, g, n_species, lmax=0, scale=1.0, workspace=None, stream=None):
    """table_bar [n_species][C] (float32) of species_embed for the gradient g
    [N][(lmax+1)^2 C] of its output: the rank-0 rows summed by species."""
    index, dtype = species.get_device(), _row_dtype(g, "g")
    _counts(n_species, lmax)
    NY = (lmax + 1) ** 2
    if species.dim() != 1 or g.dim() != 2 or g.shape[1] % NY:
        raise ValueError("species [N] and g [N][(lmax+1)^2 C] expected")
    N, C = species.shape[0], g.shape[1] // NY
    _counts(N, C)
    bar = torch.empty((n_species, C), dtype=_F32, device=index)
    need = _scratch_size(index, "fc_species_embed_vjp_workspace_size", None, N, operator.index(n_species), C)
    workspace, ws, size = _bytes(workspace, need, index)
    _check(_lib.fc_species_embed_vjp(dtype, N, n_species, lmax, C, scale,
                                     _on(species, _I32, "species", index, (N,)),
                                     _on(g, g.dtype, "g", index, (N, NY * C)), bar.data_ptr(), ws, size,
                                     stream), "fc_species_embed_vjp")
    return bar


@functools.lru_cache(maxsize=256)
def _head_desc_of(*fields):
    return HeadDesc(*fields)


def _head_desc(dtype, heads_q, heads_k, head_dim, pairs, eps):
    """Descriptor of these values.  They are looked up as plain numbers: a tensor of one element would be found by
    its identity, whatever it holds by then."""
    return _head_desc_of(dtype, operator.index(heads_q), operator.index(heads_k), head_dim, pairs, float(eps))


def _head_args(x, heads_q, gamma_q, gamma_k, pos, freq, eps):
    index, dtype = x.get_device(), _row_dtype(x, "x")
    N, H, D = _rows3(x, "x")
    _counts(N, H, D)
    px, ldx = _rows(x, "x", x.dtype, index, (N, H, D))
    if not 0 <= heads_q <= H:
        raise ValueError("heads_q %d of %d heads" % (heads_q, H))
    if (pos is None) != (freq is None):
        raise ValueError("pos and freq go together")
    R = 0 if freq is None else freq.shape[-1]
    small = (_on(gamma_q, _F32, "gamma_q", index, (D,)), _on(gamma_k, _F32, "gamma_k", index, (D,)),
             _on(pos, _F32, "pos", index, (N, 3)), _on(freq, _F32, "freq", index, (3, R)))
    return index, px, ldx, small, _head_desc(dtype, heads_q, H - heads_q, D, R, eps)


@_node_op
def head_norm_rotate(x, heads_q, gamma_q=None, gamma_k=None, pos=None, freq=None, eps=1e-6,
                     out=None, stream=None):
    """RMS norm of the heads x [N][heads][head_dim] (the first heads_q are
    queries, the rest keys; x may be a column block of a fused projection) and
    their rotation by theta_f = pos . freq[:, f] of pairs (f, f + R), with pos
    [N][3] and freq [3][R] (None: norm only).  Returns rows like x, packed."""
    index, px, ldx, small, d = _head_args(x, heads_q, gamma_q, gamma_k, pos, freq, eps)
    if out is None:
        out = x.new_empty(x.shape)
    _check(_lib.fc_head_norm_rotate(d, x.shape[0], px, ldx, *small,
                                    *_rows(out, "out", x.dtype, index, x.shape), stream),
           "fc_head_norm_rotate")
    return out


@_node_op
def head_norm_rotate_vjp(x, g, heads_q, gamma_q=None, gamma_k=None, pos=None, freq=None, eps=1e-6,
                         want=("x", "gamma", "pos"), workspace=None, stream=None):
    """(x_bar, gamma_q_bar, gamma_k_bar, pos_bar) of head_norm_rotate for the
    gradient g of its output; entries not in `want` are None, and pos_bar is
    None without positions."""
    index, px, ldx, small, d = _head_args(x, heads_q, gamma_q, gamma_k, pos, freq, eps)
    N, H, D = x.shape
    xb = x.new_empty((N, H, D)) if "x" in want else None
    gb = torch.empty((2, D), dtype=_F32, device=index) if "gamma" in want else None
    pb = torch.empty((N, 3), dtype=_F32, device=index) if "pos" in want and pos is not None else None
    need = 0 if gb is None else _scratch_size(index, "fc_head_norm_rotate_vjp_workspace_size", d, N)
    workspace, ws, size = _bytes(workspace, need, index)
    gq = None if gb is None else gb.data_ptr()
    _check(_lib.fc_head_norm_rotate_vjp(
        d, N, px, ldx, *_rows(g, "g", x.dtype, index, x.shape), *small,
        None if xb is None else xb.data_ptr(), H * D, gq, None if gb is None else gq + 4 * D,
        None if pb is None else pb.data_ptr(), ws, size, stream), "fc_head_norm_rotate_vjp")
    gqb, gkb = (None, None) if gb is None else gb.unbind(0)
    return xb, gqb, gkb, pb


@functools.lru_cache(maxsize=256)
def _attn_desc_of(*fields):
    return AttnDesc(*fields)


def _attn_desc(dtype, heads, kv_heads, head_dim, scale, cap):
    return _attn_desc_of(dtype, heads, kv_heads, head_dim, float(scale), float(cap))


def _attn_args(q, k, v, recv_ptr, send_ptr, pos, pos_send, slope, send_mask, scale, cap):
    """Device index, checked descriptor, sizes, and the arguments both directions share."""
    index, dtype = q.get_device(), _row_dtype(q, "q")
    nr, H, D = _rows3(q, "q")
    ns, KV, _ = _rows3(k, "k")
    _counts(nr, ns, H, KV, D)
    if recv_ptr.dim() != 1 or recv_ptr.shape[0] < 1:
        raise ValueError("recv_ptr shape %s" % (tuple(recv_ptr.shape),))
    if send_ptr is None:
        if nr != ns:
            raise ValueError("send_ptr is needed where senders are not the receivers")
        send_ptr = recv_ptr
    if (pos is None) != (slope is None) or (pos is None and pos_send is not None):
        raise ValueError("pos and slope go together, pos_send needs both")
    if pos is not None and pos_send is None and nr != ns:
        raise ValueError("pos_send is needed where senders are not the receivers")
    B1 = recv_ptr.shape[0]
    _counts(B1)
    args = (_on(recv_ptr, _I32, "recv_ptr", index, (B1,)), _on(send_ptr, _I32, "send_ptr", index, (B1,)),
            *_rows(q, "q", q.dtype, index, (nr, H, D)), *_rows(k, "k", q.dtype, index, (ns, KV, D)),
            *_rows(v, "v", q.dtype, index, (ns, KV, D)), _on(pos, _F32, "pos", index, (nr, 3)),
            _on(pos_send, _F32, "pos_send", index, (ns, 3)), _on(slope, _F32, "slope", index, (H,)),
            _on(send_mask, _U8, "send_mask", index, (ns,)))
    d = _attn_desc(dtype, H, KV, D, D ** -0.5 if scale is None else scale, cap)
    return index, d, (B1 - 1, nr, ns), args


def node_attention_on_tcgen05(dtype, heads, kv_heads, head_dim, n_struct, n_recv, n_send, vjp=False):
    """Whether node_attention (or its VJP) of these sizes runs on the tcgen05
    kernels, whose bounded waits device_error() reports."""
    if dtype not in _ROW_DTYPES:
        raise TypeError("rows are float32, bfloat16 or float16, got %s" % (dtype,))
    _counts(heads, kv_heads, head_dim, n_struct, n_recv, n_send)
    d = _attn_desc(_ROW_DTYPES[dtype], heads, kv_heads, head_dim, 1.0, 0.0)
    on = _lib.fc_node_attention_on_tcgen05(d, n_struct, n_recv, n_send, int(vjp))
    if on < 0:
        raise ValueError("node_attention takes no such sizes")
    return on == 1


@_node_op
def node_attention(q, k, v, recv_ptr, send_ptr=None, pos=None, pos_send=None, slope=None,
                   send_mask=None, scale=None, cap=0.0, residual=False, workspace=None, stream=None):
    """(out [n_recv][heads][head_dim], lse [n_recv][heads], out_f32) of the
    attention of q [n_recv][heads][head_dim] to k, v [n_send][kv_heads][head_dim]
    inside each structure: receivers recv_ptr[b] .. recv_ptr[b+1], senders
    send_ptr[b] .. (None: the receivers).  Scores scale q.k (scale None:
    head_dim^-1/2), capped by cap tanh(. / cap) if cap > 0, minus slope[head]
    times the distance of pos and pos_send (None: pos).  send_mask: uint8, 0
    hides a sender.  Rows without senders are 0 with lse -inf.  out_f32, which
    node_attention_vjp needs, is None unless residual (float32: it is out)."""
    index, d, sizes, args = _attn_args(q, k, v, recv_ptr, send_ptr, pos, pos_send, slope, send_mask,
                                       scale, cap)
    nr, H, D = q.shape
    out = q.new_empty((nr, H, D))
    lse = torch.empty((nr, H), dtype=_F32, device=index)
    o32, p32 = None, None
    if residual:
        if q.dtype is _F32:
            o32 = out
        else:
            o32 = torch.empty((nr, H, D), dtype=_F32, device=index)
            p32 = o32.data_ptr()
    workspace, ws, size = _bytes(workspace, _scratch_size(index, "fc_node_attention_workspace_size", d, *sizes),
                                 index)
    _check(_lib.fc_node_attention(d, *sizes, *args, out.data_ptr(), H * D, lse.data_ptr(), p32, ws, size,
                                  stream), "fc_node_attention")
    return out, lse, o32


@_node_op
def node_attention_vjp(q, k, v, out_f32, lse, g, recv_ptr, send_ptr=None, pos=None, pos_send=None,
                       slope=None, send_mask=None, scale=None, cap=0.0,
                       want=("q", "k", "v", "pos", "slope"), workspace=None, stream=None):
    """(q_bar, k_bar, v_bar, pos_bar, pos_send_bar, slope_bar) of node_attention
    for the gradient g of out, given the out_f32 (residual=True) and lse it
    returned.  Without pos_send, pos_bar holds both roles of a node and
    pos_send_bar is None; entries not in `want`, and without a bias those of
    pos and slope, are None."""
    index, d, sizes, args = _attn_args(q, k, v, recv_ptr, send_ptr, pos, pos_send, slope, send_mask,
                                       scale, cap)
    if out_f32 is None:
        raise ValueError("out_f32 is needed: node_attention(..., residual=True) returns it")
    shape = q.shape
    _, nr, ns = sizes
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    qb = q.new_empty(shape) if "q" in want else None
    kb = q.new_empty(k.shape) if "k" in want else None
    vb = q.new_empty(k.shape) if "v" in want else None
    pb = torch.empty((nr, 3), dtype=_F32, device=index) if "pos" in want and pos is not None else None
    psb = torch.empty((ns, 3), dtype=_F32, device=index) if "pos" in want and pos_send is not None else None
    sb = torch.empty((shape[1],), dtype=_F32, device=index) if "slope" in want and slope is not None else None
    workspace, ws, size = _bytes(
        workspace, _scratch_size(index, "fc_node_attention_vjp_workspace_size", d, *sizes), index)
    _check(_lib.fc_node_attention_vjp(
        d, *sizes, *args, _on(out_f32, _F32, "out_f32", index, shape), _on(lse, _F32, "lse", index, shape[:2]),
        *_rows(g, "g", q.dtype, index, shape), at(qb), at(kb), at(vb), at(pb), at(psb), at(sb), ws, size,
        stream), "fc_node_attention_vjp")
    return qb, kb, vb, pb, psb, sb
