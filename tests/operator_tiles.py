"""Which kernel instance serves a size, as the library itself chooses it (no GPU needed), and sizes that
reach every instance: tiles on SM pairs, single-CTA tiles of each width (``d``: stores in steps of 16
columns), and tiles whose K is split over a cluster. All of them end inside a tile."""
from __future__ import annotations

import ctypes

STORE, GATED, GRAD, INT8 = 0, 1, 2, 3                # the epilogues (csrc/dense.cuh)

# (T, K, N) and (T, d, F), beside those of the parity tests
MATMUL = [(19, 1184, 16), (17, 4448, 16), (17, 16, 9632), (145, 16, 4976), (17, 4016, 1296),
          (139, 304, 9776), (1337, 2064, 4112)]
FFN = [(829, 144, 7216), (135, 5536, 16), (87, 2160, 4832), (23, 4256, 1136), (6341, 1104, 160),
       (17, 16, 10896), (1663, 416, 2656), (17, 16, 1072), (2751, 16, 16), (6533, 2928, 16),
       (581, 6352, 240), (7686, 2960, 48), (1209, 1040, 4112), (4301, 1088, 1216), (17, 9712, 16),
       (1, 9488, 592)]


class _Tile(ctypes.Structure):
    _fields_ = [("pair", ctypes.c_bool), ("bn", ctypes.c_int), ("split", ctypes.c_int),
                ("direct", ctypes.c_bool)]


class Choice:
    """The library's rules: C++ functions of the shared library, by their mangled names."""

    def __init__(self, lib):
        three = ctypes.c_int * 3
        self._three = three
        self._tile = lib["_ZN3moe10dense_tileEiPA3_KiiPd"]
        self._tile.restype = _Tile
        self._tile.argtypes = [ctypes.c_int, ctypes.POINTER(three), ctypes.c_int,
                               ctypes.POINTER(ctypes.c_double)]
        self._few = lib["_ZN3moe13few_rows_winsEiiii"]
        self._few.restype = ctypes.c_bool
        self._few.argtypes = [ctypes.c_int] * 4

    def tile(self, epi, *mnk):
        """The instance's name and the estimated cycles of a launch of these products."""
        cost = ctypes.c_double()
        t = self._tile(epi, (self._three * len(mnk))(*[self._three(*m) for m in mnk]), len(mnk),
                       ctypes.byref(cost))
        if t.pair:
            name = "pair"
        elif t.split > 1:
            name = f"split{t.bn}x{t.split}"
        else:
            width = 256 if t.bn > 128 else 128 if (epi == GATED or t.bn > 64) else 64
            name = f"single{width}" + ("d" if t.direct else "")
        return name, cost.value

    def one(self, epi, T, N, K):
        return "few" if self._few(epi, T, N, K) else self.tile(epi, (T, N, K))[0]

    def matmul(self, T, K, N):
        return {"int8 " + self.one(INT8, T, N, K)}

    def ffn(self, T, d, F):
        got = {"gated " + self.one(GATED, T, F, d), "down " + self.one(STORE, T, d, F),
               "gradient of the activation " + self.tile(GRAD, (T, F, d))[0]}
        products = [(T, d, 2 * F), (2 * F, d, T), (d, F, T)]
        together, c3 = self.tile(STORE, *products)
        alone, c1 = self.tile(STORE, products[0])
        rest, c2 = self.tile(STORE, *products[1:])
        if c3 <= c1 + c2 + 5000:                     # (a further launch's cost, csrc/gated_ffn.cu)
            return got | {"three products " + together}
        return got | {"dx " + alone, "weight gradients " + rest}
