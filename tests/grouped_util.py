"""Which form of the grouped kernel a shape gets (the library's own choice, host arithmetic)."""
import ctypes

import q4_q8_int8_amd as mmq


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("P", "E", "N", "K", "q_rows", "per_row")]


def grouped_form(P: int, E: int, N: int, K: int, compute_units: int = 256) -> str:
    """N weight rows (a gated product: its packed rows) of E matrices, P pairs."""
    fn = mmq._lib["_ZN3mmq12grouped_formERKNS_12GroupedShapeEl"]
    fn.restype = ctypes.c_int
    s = Shape(P, E, N, K, P, 1)
    return ("wide", "narrow", "split2", "split4")[fn(ctypes.byref(s), ctypes.c_int64(compute_units))]


def rows_in_32(n: int) -> int:
    """The first of an expert's n rows, up to its last tile where that has 16 rows or fewer (which the forms
    of 32 rows sum in another order)."""
    return n // 32 * 32 if n % 32 <= 16 else n
