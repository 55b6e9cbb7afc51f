"""C signatures of the entry points that kv.py calls (include/exact_attention.h)."""
import ctypes

_c = ctypes
_p, _i, _l, _f, _z = _c.c_void_p, _c.c_int, _c.c_longlong, _c.c_float, _c.c_size_t

FA_ROPE_INTERLEAVED = 1
FA_ROPE_INVERSE = 2

SIGNATURES = {
    "fa_rope": (_i, [_p, _p, _p, _p, _i, _p, _p, _p, _p, _i, _i, _i, _i, _p, _l, _p, _i, _i, _f,
                     _p]),
    "fa_rope_axes": (_i, [_p, _p, _p, _p, _i, _p, _p, _p, _p, _i, _i, _i, _i, _p, _i, _l, _l, _p, _p, _i, _i,
                          _f, _p]),
    "fa_page_plan": (_i, [_p, _p, _p, _i, _p, _i, _p, _i, _i, _i, _p, _p, _p, _p, _p, _p]),
    "fa_kv4_cache_bytes": (_z, [_i, _i, _i, _i]),
    "fa_kv4_append": (_i, [_p, _l, _l, _p, _l, _l, _p, _i, _i, _p, _i, _i, _i, _f, _f, _p]),
    "fa_kv4_read": (_i, [_p, _i, _i, _p, _p, _p, _i, _i, _i, _f, _f, _p]),
    "fa_kv4_fwd": (_i, [_p, _l, _l, _p, _i, _i, _p, _i, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f,
                        _i, _f, _f, _p, _z, _p, _p]),
    "fa_kv4_fwd_workspace_bytes": (_z, [_i, _i, _i, _i, _i, _i]),
    "fa_tree_plan": (_i, [_p, _p, _p, _i, _i, _i, _p, _p, _p]),
    "fa_tree_accept": (_i, [_p, _p, _i, _p, _p, _p, _p, _p, _p, _p, _i, _p, _i, _p, _i, _i, _i, _p, _p, _p, _p,
                            _p, _p, _p]),
    "fa_kv4_move": (_i, [_p, _i, _i, _i, _i, _i, _p, _p, _p, _p, _i, _i, _p]),
    "fa_kv4_tree_fwd": (_i, [_p, _l, _l, _p, _i, _i, _p, _i, _p, _p, _p, _i, _p, _p, _i, _i, _i, _i, _i, _i, _f,
                             _f, _f, _p, _z, _p, _p]),
    "fa_kv4_tree_fwd_workspace_bytes": (_z, [_i, _i, _i, _i, _i, _i]),
}
