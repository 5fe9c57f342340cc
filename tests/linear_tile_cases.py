"""Sizes of the dense projection (one weight matrix, a workspace given, 256 CUs) with the tiles that they run in.

(M, N, K, tile kind, slices of the reduction, rows streamed behind the tiles).  Kinds: 0 256x256, 1 256x128, 2 128x128,
3 64x128.  Every kind comes with rows that are whole 16-byte pieces and with odd ones, and with its reduction split.
"""
CASES = [(3001, 4101, 72, 0, 1, 0), (3000, 4104, 72, 0, 1, 0), (2000, 2050, 8200, 0, 3, 0),
         (1500, 4101, 520, 1, 1, 0), (1500, 4104, 520, 1, 1, 0), (1500, 1301, 4104, 1, 3, 0),
         (1500, 4101, 72, 2, 1, 0), (1500, 4104, 72, 2, 1, 0), (4099, 131, 4104, 2, 3, 0),
         (1100, 1031, 72, 3, 1, 0), (1100, 1032, 72, 3, 1, 0), (400, 771, 12296, 3, 5, 0), (1795, 1029, 2056, 3, 1, 3)]
